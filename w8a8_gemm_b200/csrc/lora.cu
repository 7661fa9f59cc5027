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
// Three kernels, and one for the forward pass of few rows:
//   contract  [rows] x [C] -> [rows] x R: t (rows of A) and dt (columns of B);
//   expand    [rows] x R -> [rows] x [C] added to base: y and dx;
//   outer     [rows] x [C], [rows] x R -> [C] x R: dB and dA.
// All are bound by the rows' traffic (at rank 64 a row element that is read
// and written, four bytes, meets 128 flop).  Sums are fp32; the small operand t
// (dt) enters the second product as bf16 where the result is rounded to bf16
// anyway, or split into three bf16 terms (24 significant bits) where the result
// stays fp32; dx beside fp32 gradients takes two of dt's.
//
// Times here are of replayed graphs of ten calls on one input, which leave out the
// host and find in L2 what fits; a call with new inputs takes up to a tenth more.
#include <cooperative_groups.h>
#include <cuda.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include <type_traits>

#include "bf16.cuh"
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
// (Once per batch: 4 us up to 333 rows, 5.3 for 1501, 9 for 8858 of two adapters, 16
// of 64, 59 for 100,000; through ctypes a call takes 7 at least.)
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
  // Before a wait for a free stage: whoever frees it may itself be waiting for
  // a stage whose copies have landed without being announced, so nothing is
  // held back unless the stage is free already.
  __device__ __forceinline__ void before_wait(int lane, uint64_t *bar, uint32_t parity) {
    if (older == nullptr && newer == nullptr) return;
    bool ready = lane == 0 ? mbar_try_wait(bar, parity) : true;
    if (!__all_sync(~0u, ready)) catch_up(lane);
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

template <bool F32>
__device__ __forceinline__ void store_grad(void *out, int64_t at, float v) {
  if constexpr (F32)
    static_cast<float *>(out)[at] = v;
  else
    static_cast<__nv_bfloat16 *>(out)[at] = __float2bfloat16_rn(v);
}

// v as bf16 (nearest even), or as three bf16 values whose sum is v with its 24
// bits (in steps of 2^-133, the smallest bf16 number), packed in pairs.  Three are
// cut off towards zero, all of v's sign, and none is zero unless v is (a place
// that would be holds 2^-40 of v, far below its last bit): an infinite factor then
// meets terms of one sign, and neither 0 times infinity nor infinity less infinity
// comes up that the product itself does not have.  For the same reason an infinite
// or NaN v is one in every place.
__device__ __forceinline__ void three_terms(float v, uint32_t (&t)[3]) {
  const uint32_t u = __float_as_uint(v), e = u & 0x7F800000u;
  if (e == 0x7F800000u) {
    t[0] = t[1] = t[2] = (u >> 16) | ((u & 0x007FFFFFu) != 0 ? 0x40u : 0u);
    return;
  }
  const uint32_t least =
      e == 0 ? 0u : (u & 0x80000000u) | (e > (40u << 23) ? e - (40u << 23) : 0x00010000u);
#pragma unroll
  for (int s = 0; s < 3; ++s) {
    const uint32_t w = __float_as_uint(v) & 0xFFFF0000u;
    v -= __uint_as_float(w);
    t[s] = ((w & 0x7FFF0000u) != 0 ? w : least) >> 16;
  }
}
template <int TERMS>
__device__ __forceinline__ void split_terms(float4 v, uint2 (&out)[TERMS]) {
  static_assert(TERMS == 1 || TERMS == 3, "bf16 or 24 bits");
  if constexpr (TERMS == 1) {
    out[0] = make_uint2(bf16x2(v.x, v.y), bf16x2(v.z, v.w));
  } else {
    uint32_t x[3], y[3], z[3], w[3];
    three_terms(v.x, x);
    three_terms(v.y, y);
    three_terms(v.z, z);
    three_terms(v.w, w);
#pragma unroll
    for (int s = 0; s < 3; ++s) out[s] = make_uint2(x[s] | y[s] << 16, z[s] | w[s] << 16);
  }
}

// ------------------------------------------------------------------- contract
// t[m][j] = sum_c in[m][c] W(j, c), W(j, c) = w[a][j][c] (TRANS false: A), or
// dt[m][j] = scale[a] sum_c in[m][c] W(j, c), W(j, c) = w[a][c][j] (TRANS true:
// B, an operand whose rows run along the contraction).  One block per row tile and
// slice of the contracted dimension: TMA brings the tile's rows as a box, 64
// columns a stage, where they are neighbours (else four warps take 32 each, as a
// box or by copies), and the weight's box beside them; one thread issues
// tcgen05.mma (M = 128, N = RT, sums in tensor memory), so that reading the rows
// costs the SM next to no instructions.  The blocks of a cluster hold the slices
// of one tile and add their partial sums through distributed shared memory in a
// fixed order.  The operand of the second products is stored as bf16 terms by
// tile, 128 rows each with zeros past the tile's last: scale t (forward, beside t by
// row in fp32), or dt and t (backward).  Bound by the rows' way from HBM: 8858 x
// 6144, rank 64, 113 MB in 30 us from a cold L2 (profiler; tensor pipe 11%, issue
// 13%).
struct ContractArgs {
  const uint16_t *in;  // as tm_in
  int64_t ld;
  const float *scale;  // nullptr: 1
  const int32_t *plan;
  float *t;               // [M][R]; forward writes it, backward reads it
  uint16_t *v;            // [TERMS][max_tiles][128][R]: scale t (forward), dt
  uint16_t *vt;           // backward: t, laid out as v
  int64_t M, max_tiles;
  int32_t C, R, L;
  int *status;
};

// Warps: 0 TMA, 1 products, 4 .. 7 copies of scattered rows (one warp by itself
// takes 128 clocks a copy instruction: 1501 rows of 1536 took 19 us); all of them
// store.
constexpr int kContractThreads = 256, kCopyWarps = 4;

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

// TRANS false: the forward pass, true: the backward pass.
template <int RT, bool TRANS, int TERMS>
__global__ void __launch_bounds__(kContractThreads)
    lora_contract_kernel(const __grid_constant__ CUtensorMap tm_in,
                         const __grid_constant__ CUtensorMap tm_in32,
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
      mbar_init(&full[s], run ? 1 : 1 + kCopyWarps);
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
      if (lane == 0) {
        const int first = rec[4];
        const uint32_t bytes = (run ? S::kIn : 0) + S::kW;
        uint32_t armed = 0, armed_parity = 0;
        for (int step = 0; step < steps; ++step) {
          const int st = step % STAGES;
          const uint32_t phase = (step / STAGES) & 1;
          uint8_t *in = smem + st * S::kStage;
          const int c0 = c_lo + step * 64;
          if (!bounded_wait(&empty[st], phase ^ 1, abort_flag, p.status, SQ_ERR_DEVICE_TIMEOUT))
            break;
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
        // never leave with a copy in flight into this block's shared memory
        for (int s = 0; s < STAGES; ++s)
          if (armed & (1u << s)) mbar_wait(&full[s], (armed_parity >> s) & 1u, kBoundedWaitNs);
      }
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
    } else if (warp >= 4 && !run) {
      // ------------------------------------------------- scattered rows: copies
      // This warp's 32 rows: a box where they are neighbours (rows ascend within a
      // tile), else four a copy instruction.
      const int first = (warp - 4) * 32, c = lane & 7;
      const int row0 = rec[4 + first];
      const bool box = first + 32 <= count && rec[4 + first + 31] - row0 == 31;
      int32_t rows[8];
#pragma unroll
      for (int i = 0; i < 8; ++i) rows[i] = rec[4 + first + i * 4 + (lane >> 3)];
      LateArrival late;
      for (int step = 0; step < steps; ++step) {
        const int st = step % STAGES;
        const uint32_t phase = (step / STAGES) & 1;
        late.before_wait(lane, &empty[st], phase ^ 1);
        bool ok = true;
        if (lane == 0)
          ok = bounded_wait(&empty[st], phase ^ 1, abort_flag, p.status, SQ_ERR_DEVICE_TIMEOUT);
        if (!__shfl_sync(~0u, ok, 0)) break;
        if (box) {
          if (lane == 0) {
            mbar_arrive_expect_tx(&full[st], 4096);
            tma_load_2d(smem + st * S::kStage + first * 128, &tm_in32, &full[st],
                        c_lo + step * 64, row0);
          }
          continue;
        }
        const int col = c_lo + step * 64 + c * 8;
        const bool in_cols = col < p.C;
        const uint32_t to = smem_u32(smem + st * S::kStage);
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          const int r = first + i * 4 + (lane >> 3);
          if (r < count)
            cp_async16(to + swz128(r, c), p.in + rows[i] * p.ld + (in_cols ? col : 0), in_cols);
        }
        cp_async_commit();
        late.push(lane, &full[st]);
      }
      late.catch_up(lane);
      cp_async_wait<0>();
    }
    const bool ok = bounded_wait(done, 0, abort_flag, p.status, SQ_ERR_DEVICE_TIMEOUT);
    tc_fence_after();
    // nothing reads or fills the stages any more
    __syncthreads();

    // partial sums -> shared memory -> sum over the slices
    float *part = reinterpret_cast<float *>(smem);
    constexpr int PS = S::kPartRow;
    const int quarter = warp & 3;  // TMEM lanes this warp may read
#pragma unroll
    for (int c0 = 0; c0 < RT / 2; c0 += 32) {
      const int c = (warp >> 2) * (RT / 2) + c0;
      uint32_t r[32];
      __syncwarp();
      tmem_ld_32x32b_x32(tmem + c + (static_cast<uint32_t>(quarter * 32) << 16), r);
      tmem_ld_wait();
      float *to = part + (quarter * 32 + lane) * PS + c;
#pragma unroll
      for (int j = 0; j < 32; j += 4)
        *reinterpret_cast<uint4 *>(to + j) =
            steps > 0 ? make_uint4(r[j], r[j + 1], r[j + 2], r[j + 3]) : make_uint4(0, 0, 0, 0);
    }
    if (slices > 1) cluster.sync(); else __syncthreads();
    const float f = p.scale[bin];
    const int quads = p.R / 4;
    const int total = ok ? kTileRows * quads : 0;
    for (int e = rank * kContractThreads + threadIdx.x; e < total;
         e += slices * kContractThreads) {
      const int r = e / quads, j = (e - r * quads) * 4;
      float4 s = make_float4(0.0f, 0.0f, 0.0f, 0.0f), t = s;
      const int row = rec[4 + r];
      const int64_t at = static_cast<int64_t>(row) * p.R + j;
      if (r < count) {
        s = slices > 1 ? cluster_sum(cluster, part, 0, slices - 1, [&](int) { return r * PS + j; })
                       : *reinterpret_cast<const float4 *>(part + r * PS + j);
        if constexpr (TRANS) {
          t = *reinterpret_cast<const float4 *>(p.t + at);
        } else if (store_ok(p.status, row >= 0 && row < p.M && j + 4 <= p.R)) {
          *reinterpret_cast<float4 *>(p.t + at) = s;
        }
        s = make_float4(f * s.x, f * s.y, f * s.z, f * s.w);
      }
      const int64_t place = static_cast<int64_t>(blockIdx.x) * kTileRows + r;
      if (!store_ok(p.status, place < p.max_tiles * kTileRows)) continue;
      uint2 d[TERMS];
      split_terms<TERMS>(s, d);
#pragma unroll
      for (int q = 0; q < TERMS; ++q)
        *reinterpret_cast<uint2 *>(p.v + (q * p.max_tiles * kTileRows + place) * p.R + j) = d[q];
      if constexpr (TRANS) {
        split_terms<TERMS>(t, d);
#pragma unroll
        for (int q = 0; q < TERMS; ++q)
          *reinterpret_cast<uint2 *>(p.vt + (q * p.max_tiles * kTileRows + place) * p.R + j) = d[q];
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

// ------------------------------------------------------------- forward, few rows
// t and y of a few rows (single tokens of many requests) in one kernel: the
// weights of the adapters in use are nearly all that is read, and what counts is
// the chain of latencies, not the rate of the products: warp-level mma (16 rows)
// takes its operands straight from global memory, with no stage to fill.  A
// cluster of eight blocks per tile: each block multiplies its slice of K, the
// blocks exchange t through distributed shared memory, and each writes its slice
// of the columns, whose weights and base came meanwhile.
struct FewArgs {
  const uint16_t *x, *A, *B;
  const float *scale;
  const int32_t *plan;
  const void *base;
  void *y;
  float *t;
  int64_t ldx, ld_base, ldy, M;
  int32_t N, K, R, L;
  int *status;
};

constexpr int kFewThreads = 256, kFewWarps = kFewThreads / 32, kFewCluster = 8, kFewRows = 16;

template <int RT, int TERMS>
struct FewSmem {
  static constexpr int kPart = kFewRows * RT;     // floats
  static constexpr int kTermRow = RT + 8;         // bf16
  static constexpr int kBytes =
      (kFewWarps + 1) * kPart * 4 + TERMS * kFewRows * kTermRow * 2;
};

// D (16 x 8 fp32) += A (16 x 16 bf16) B (16 x 8 bf16).  Lane 4 g + t has rows g
// and g + 8 of A, column g of B, and of D the columns 2 t, 2 t + 1 of rows g and
// g + 8.  Which terms of the contraction a register holds is free as long as A
// and B agree: here a lane's 16 bytes are two steps' worth.
__device__ __forceinline__ void mma_rows(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2,
                                         uint32_t a3, uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, "
      "{%8, %9}, {%0, %1, %2, %3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
__device__ __forceinline__ void mma_rows_32(float (&d)[4], const uint4 &lo, const uint4 &hi,
                                            const uint4 &w) {
  mma_rows(d, lo.x, hi.x, lo.y, hi.y, w.x, w.y);
  mma_rows(d, lo.z, hi.z, lo.w, hi.w, w.z, w.w);
}
// Two neighbouring values of y's type.
template <bool F32>
__device__ __forceinline__ float2 load_pair(const void *p, int64_t at) {
  if constexpr (F32) return *reinterpret_cast<const float2 *>(static_cast<const float *>(p) + at);
  const uint32_t w = *reinterpret_cast<const uint32_t *>(static_cast<const uint16_t *>(p) + at);
  return make_float2(bf16_lo(w), bf16_hi(w));
}
template <bool F32>
__device__ __forceinline__ void store_pair(void *p, int64_t at, float2 v) {
  if constexpr (F32)
    *reinterpret_cast<float2 *>(static_cast<float *>(p) + at) = v;
  else
    *reinterpret_cast<uint32_t *>(static_cast<uint16_t *>(p) + at) = bf16x2(v.x, v.y);
}

template <int RT, bool F32>
__global__ void __launch_bounds__(kFewThreads) lora_few_kernel(const FewArgs p) {
  constexpr int TERMS = F32 ? 3 : 1, STEPS = RT / 32;
  using S = FewSmem<RT, TERMS>;
  extern __shared__ float few_sh[];
  float *sums = few_sh;                          // [warps][16][R]
  float *part = few_sh + kFewWarps * S::kPart;   // [16][R], this block's slice of K
  uint16_t *terms = reinterpret_cast<uint16_t *>(part + S::kPart);  // [TERMS][16][kTermRow]
  cg::cluster_group cluster = cg::this_cluster();
  const int rank = static_cast<int>(cluster.block_rank());
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, t8 = (lane & 3) * 8;
  const int R = p.R, quads = R / 4;
  for (int e = threadIdx.x; e < TERMS * kFewRows * S::kTermRow / 2; e += kFewThreads)
    reinterpret_cast<uint32_t *>(terms)[e] = 0;  // columns past R
  grid_dependency_wait();
  grid_dependency_launch();
  // the blocks of a cluster share their tile and so their way through the kernel
  if (!plan_fits(p.plan, p.M, p.L, p.status) || static_cast<int>(blockIdx.x) >= p.plan[3]) return;
  const int32_t *rec = p.plan + plan_recs_at(p.L) + static_cast<int64_t>(blockIdx.x) * kRecWords;
  const int bin = rec[0], count = rec[1];
  const int32_t *row = rec + 4;  // past the last: the first again
  const int cols = (p.N / 8 + kFewCluster - 1) / kFewCluster * 8;
  const int c_lo = rank * cols, c_hi = c_lo + cols < p.N ? c_lo + cols : p.N;
  if (bin == p.L) {  // no adapter: y is base
    if (p.base == p.y) return;
    for (int m = warp; m < count; m += kFewWarps)
      for (int c = c_lo + lane * 2; c < c_hi; c += 64)
        if (store_ok(p.status, row[m] >= 0 && row[m] < p.M && c + 2 <= p.N))
          store_pair<F32>(p.y, row[m] * p.ldy + c,
                          p.base ? load_pair<F32>(p.base, row[m] * p.ld_base + c)
                                 : make_float2(0.0f, 0.0f));
    return;
  }
  const int span = (p.K / 8 + kFewCluster - 1) / kFewCluster * 8;
  const int k_lo = rank * span, k_hi = k_lo + span < p.K ? k_lo + span : p.K;
  const uint16_t *A = p.A + static_cast<int64_t>(bin) * R * p.K;
  const uint16_t *B = p.B + static_cast<int64_t>(bin) * p.N * R;
  const float f = p.scale[bin];

  for (int m0 = 0; m0 < count; m0 += kFewRows) {
    // t: a warp takes every eighth run of 32 columns, for all ranks
    const int64_t r0 = row[m0 + g], r1 = row[m0 + g + 8];
    const uint4 none = make_uint4(0, 0, 0, 0);
    float acc[RT / 8][4];
#pragma unroll
    for (int n = 0; n < RT / 8; ++n) acc[n][0] = acc[n][1] = acc[n][2] = acc[n][3] = 0.0f;
    for (int k = k_lo + warp * 32; k < k_hi; k += kFewWarps * 32) {
      const int kk = k + t8;  // K % 8 == 0
      const bool in = kk < k_hi;
      const uint4 lo = in ? *reinterpret_cast<const uint4 *>(p.x + r0 * p.ldx + kk) : none;
      const uint4 hi = in ? *reinterpret_cast<const uint4 *>(p.x + r1 * p.ldx + kk) : none;
      uint4 w[RT / 8];
#pragma unroll
      for (int n = 0; n < RT / 8; ++n) {
        w[n] = none;
        if (in && n * 8 < R)
          w[n] = *reinterpret_cast<const uint4 *>(A + static_cast<int64_t>(n * 8 + g) * p.K + kk);
      }
#pragma unroll
      for (int n = 0; n < RT / 8; ++n)
        if (n * 8 < R) mma_rows_32(acc[n], lo, hi, w[n]);
    }
    float *mine = sums + warp * kFewRows * R + g * R + t8 / 4;
#pragma unroll
    for (int n = 0; n < RT / 8; ++n)
      if (n * 8 < R) {
        *reinterpret_cast<float2 *>(mine + n * 8) = make_float2(acc[n][0], acc[n][1]);
        *reinterpret_cast<float2 *>(mine + 8 * R + n * 8) = make_float2(acc[n][2], acc[n][3]);
      }
    // the first columns' weights and base come while the sums meet
    int c = c_lo + warp * 8;
    uint4 w[STEPS];
    float2 b0, b1;
    auto load = [&]() {
      if (c >= c_hi) return;
#pragma unroll
      for (int q = 0; q < STEPS; ++q)
        w[q] = q * 32 + t8 < R ? *reinterpret_cast<const uint4 *>(
                                     B + static_cast<int64_t>(c + g) * R + q * 32 + t8)
                               : none;
      b0 = b1 = make_float2(0.0f, 0.0f);
      if (p.base != nullptr) {
        if (m0 + g < count) b0 = load_pair<F32>(p.base, r0 * p.ld_base + c + t8 / 4);
        if (m0 + g + 8 < count) b1 = load_pair<F32>(p.base, r1 * p.ld_base + c + t8 / 4);
      }
    };
    load();
    __syncthreads();
    for (int e = threadIdx.x; e < kFewRows * quads; e += kFewThreads) {
      float4 s = reinterpret_cast<const float4 *>(sums)[e];
#pragma unroll
      for (int v = 1; v < kFewWarps; ++v) {
        const float4 u = reinterpret_cast<const float4 *>(sums)[v * kFewRows * quads + e];
        s = make_float4(s.x + u.x, s.y + u.y, s.z + u.z, s.w + u.w);
      }
      reinterpret_cast<float4 *>(part)[e] = s;
    }
    cluster.sync();
    for (int e = threadIdx.x; e < kFewRows * quads; e += kFewThreads) {
      const int m = e / quads, j = (e - m * quads) * 4;
      if (m0 + m >= count) break;
      float4 s = cluster_sum(cluster, part, 0, kFewCluster - 1, [&](int) { return e * 4; });
      const int64_t r = row[m0 + m];
      if (e % kFewCluster == rank && store_ok(p.status, r >= 0 && r < p.M && j + 4 <= R))
        *reinterpret_cast<float4 *>(p.t + r * R + j) = s;
      uint2 d[TERMS];
      split_terms<TERMS>(make_float4(f * s.x, f * s.y, f * s.z, f * s.w), d);
#pragma unroll
      for (int q = 0; q < TERMS; ++q)
        *reinterpret_cast<uint2 *>(terms + (q * kFewRows + m) * S::kTermRow + j) = d[q];
    }
    cluster.sync();  // the terms are there, and the other blocks have read this one's sums

    // y: a warp takes every eighth run of 8 columns
    while (c < c_hi) {
      float d[4] = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
      for (int v = TERMS - 1; v >= 0; --v)
#pragma unroll
        for (int q = 0; q < STEPS; ++q)
          if (q * 32 < R) {
            const uint16_t *at = terms + (v * kFewRows + g) * S::kTermRow + q * 32 + t8;
            mma_rows_32(d, *reinterpret_cast<const uint4 *>(at),
                        *reinterpret_cast<const uint4 *>(at + 8 * S::kTermRow), w[q]);
          }
      const int64_t to = c + t8 / 4;
      auto fits = [&](int64_t r) { return r >= 0 && r < p.M && to + 2 <= p.N; };
      if (m0 + g < count && store_ok(p.status, fits(r0)))
        store_pair<F32>(p.y, r0 * p.ldy + to, make_float2(b0.x + d[0], b0.y + d[1]));
      if (m0 + g + 8 < count && store_ok(p.status, fits(r1)))
        store_pair<F32>(p.y, r1 * p.ldy + to, make_float2(b1.x + d[2], b1.y + d[3]));
      c += kFewWarps * 8;
      load();
    }
  }
}

// --------------------------------------------------------------------- expand
// out[m][c] = base[m][c] + sum_j v[m][j] W(j, c); W(j, c) = w[a][c][j] (TRANS
// false: B, v = scale t) or w[a][j][c] (TRANS true: A, v = dt); v as TERMS bf16
// terms by tile.  Persistent blocks, one per SM, take equal shares of the units
// (row tile, slab of 256 bytes of columns), neighbouring slabs of a tile in a
// row.  Per unit TMA brings base and the weight slab into a stage, one thread
// issues the products (M = 128 rows, sums in tensor memory, two buffers), and
// eight warps add the sums into base where it stands in the stage and store it
// from there, by TMA where a warp's 32 rows are neighbours.  On its way through
// the SM an element meets one 16-byte shared load and store and an addition:
// with the products on the warp-level path, whose operands pass through the
// same load pipe, that pipe was the bound (8858 x 6144, rank 64: 59 us).
// Where a tile's rows are not neighbours, four warps take 32 rows of base each, as
// boxes or by copies, and begin before the contraction has ended (1501 ragged
// rows, 1536 -> 2304 in fp32: 18.9 us with the contraction; 21.0 when they wait
// for it, 25.7 with two warps), on SMs that no block of the contraction holds any
// more: the two together need more shared memory than an SM has.  Rows without
// an adapter are copied from base (left alone when out is base).  8858 x 6144, rank 64, bf16: 218
// MB in 40.5 us from a cold L2 (profiler), 5.4 TB/s.
struct ExpandArgs {
  const int32_t *plan;
  const void *base;    // nullptr: 0
  int64_t ld_base;
  void *out;
  int64_t ld_out;
  int64_t M, max_tiles;
  int32_t C, R, L;
  int *status;
};
struct ExpandMaps {
  CUtensorMap base, base32, out, w, v;  // rows of a box: 128, 32, 32
};

constexpr int kExpandWarps = 8;                            // adding and storing
constexpr int kExpandThreads = 64 + 32 * (kExpandWarps + kCopyWarps);  // and producer, MMA

template <int RT, bool F32, int TERMS>
struct ExpandSmem {
  static constexpr int kTerms = TERMS;
  static constexpr int kSlab = F32 ? 64 : 128;  // columns of a unit
  static constexpr int kBase = kTileRows * 256;
  static constexpr int kW = kSlab * RT * 2;
  static constexpr int kStage = kBase + kW;
  static constexpr int kA = kTerms * kTileRows * RT * 2;
  static constexpr int kABufs = kA <= 48 * 1024 ? 2 : 1;
  static constexpr int kFit = (226 * 1024 - kABufs * kA) / kStage;
  static constexpr int kStages = kFit > 4 ? 4 : kFit;
  static constexpr int kAAt = kStages * kStage;
  static constexpr int kBars = kAAt + kABufs * kA;
  static constexpr int kBytes = kBars + (2 * kStages + 9) * 8 + kStages * 4 + 16 + 1024;
  static_assert(kStages >= 2, "one unit ahead at least");
  static_assert(kBytes <= 232448, "dynamic shared memory above the per-block limit");
};

enum { kUnitNone = 1, kUnitFirst = 2, kUnitLast = 4, kUnitEnd = 8 };

// A block's walk over its units; every role makes the same one.  Units of rows
// without an adapter are left out when out is base.
struct Units {
  const int32_t *recs;
  int slabs, tile, slab, left;
  __device__ __forceinline__ void init(const int32_t *plan, int tiles, int L, int n_slabs) {
    recs = plan + plan_recs_at(L);
    slabs = n_slabs;
    const int64_t units = static_cast<int64_t>(tiles) * n_slabs;
    const int64_t lo = units * blockIdx.x / gridDim.x;
    left = static_cast<int>(units * (blockIdx.x + 1) / gridDim.x - lo);
    tile = static_cast<int>(lo / n_slabs);
    slab = static_cast<int>(lo - static_cast<int64_t>(tile) * n_slabs);
  }
  // slabs of the current tile that are this block's
  __device__ __forceinline__ int here() const { return left < slabs - slab ? left : slabs - slab; }
  __device__ __forceinline__ void next_tile() {
    left -= here();
    slab = 0;
    ++tile;
  }
  __device__ __forceinline__ const int32_t *rec(int t) const {
    return recs + static_cast<int64_t>(t) * kRecWords;
  }
};

template <int RT, bool TRANS, bool F32, int TERMS>
__global__ void __launch_bounds__(kExpandThreads, 1)
    lora_expand_kernel(const __grid_constant__ ExpandMaps maps, const ExpandArgs p) {
  using S = ExpandSmem<RT, F32, TERMS>;
  constexpr int STAGES = S::kStages, SLAB = S::kSlab, E = F32 ? 4 : 2;
  constexpr int BOX = 128 / E;  // columns of a 128-byte box
  extern __shared__ uint8_t smem_raw[];
  uint8_t *smem = reinterpret_cast<uint8_t *>(
      (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~static_cast<uintptr_t>(1023));
  uint64_t *full = reinterpret_cast<uint64_t *>(smem + S::kBars);
  uint64_t *empty = full + STAGES;
  uint64_t *acc_full = empty + STAGES;
  uint64_t *acc_empty = acc_full + 2;
  uint64_t *a_full = acc_empty + 2;
  uint64_t *a_empty = a_full + 2;
  uint64_t *done = a_empty + 2;
  volatile int *meta = reinterpret_cast<volatile int *>(done + 1);  // [STAGES]
  uint32_t *tmem_slot = reinterpret_cast<uint32_t *>(done + 1) + STAGES;
  volatile int *abort_flag = reinterpret_cast<volatile int *>(tmem_slot + 1);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  constexpr int kTimeout = SQ_ERR_DEVICE_TIMEOUT;

  if (threadIdx.x == 0) {
    for (int s = 0; s < STAGES; ++s) {
      mbar_init(&full[s], 1 + kCopyWarps);     // producer, copying warps
      mbar_init(&empty[s], kExpandWarps + 1);  // storing warps, MMA issuer
    }
    for (int b = 0; b < 2; ++b) {
      mbar_init(&acc_full[b], 1);
      mbar_init(&acc_empty[b], kExpandWarps);
      mbar_init(&a_full[b], 1);
      mbar_init(&a_empty[b], 1);
    }
    mbar_init(done, 1);
    *abort_flag = 0;
    fence_mbar_init();
    prefetch_tmap(&maps.base);
    prefetch_tmap(&maps.w);
    prefetch_tmap(&maps.v);
    prefetch_tmap(&maps.out);
  }
  if (warp == 1) {
    tmem_alloc(tmem_slot, 2 * SLAB);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;

  // base, weights and plan were complete before the kernel ahead of this one
  // began; only its own output, v, has to be waited for
  const bool fits = plan_fits(p.plan, p.M, p.L, p.status);
  Units u;
  u.init(p.plan, fits ? p.plan[3] : 0, p.L, (p.C + SLAB - 1) / SLAB);
  const bool has_base = p.base != nullptr, in_place = p.base == p.out;
  if (warp != 0 && warp < 2 + kExpandWarps) {
    grid_dependency_wait();
    if constexpr (TRANS) grid_dependency_launch();  // the outer products run beside
  }

  if (warp == 0) {
    // ------------------------------------------------------------ producer
    uint32_t armed = 0, armed_parity = 0;
    int step = 0, a_tiles = 0;
    bool ok = true, waited = false;
    int pending_tile[STAGES], pending = 0;  // tiles met before v may be read
    // v of a tile -> its buffer
    auto load_v = [&](int tile) {
      const int b = a_tiles % S::kABufs;
      if (!bounded_wait(&a_empty[b], ((a_tiles / S::kABufs) & 1) ^ 1, abort_flag, p.status,
                        kTimeout))
        return false;
      mbar_arrive_expect_tx(&a_full[b], S::kA);
#pragma unroll
      for (int s = 0; s < S::kTerms; ++s)
#pragma unroll
        for (int h = 0; h < RT / 64; ++h)
          tma_load_3d(smem + S::kAAt + b * S::kA + (s * (RT / 64) + h) * 16384, &maps.v,
                      &a_full[b], h * 64, tile * kTileRows, s);
      ++a_tiles;
      return true;
    };
    auto catch_up = [&]() {
      grid_dependency_wait();
      waited = true;
      for (int i = 0; i < pending && ok; ++i) ok = load_v(pending_tile[i]);
    };
    if (lane == 0) {
      for (; u.left > 0 && ok; u.next_tile()) {
        const int32_t *rec = u.rec(u.tile);
        const int4 h = *reinterpret_cast<const int4 *>(rec);
        const int first = rec[4];
        const bool none = h.x >= p.L, run = h.w != 0;
        if (none && in_place) continue;
        const int n = u.here();
        for (int i = 0; i < n && ok; ++i, ++step) {
          if (!waited && step == STAGES) catch_up();
          const int st = step % STAGES;
          const uint32_t phase = (step / STAGES) & 1;
          ok = ok && bounded_wait(&empty[st], phase ^ 1, abort_flag, p.status, kTimeout);
          if (!ok) break;
          meta[st] = (none ? kUnitNone : 0) | (i == 0 ? kUnitFirst : 0) |
                     (i == n - 1 ? kUnitLast : 0);
          const bool box = has_base && run;
          mbar_arrive_expect_tx(&full[st], (box ? S::kBase : 0) + (none ? 0 : S::kW));
          uint8_t *to = smem + st * S::kStage;
          const int c0 = (u.slab + i) * SLAB;
          if (box) {
            tma_load_2d(to, &maps.base, &full[st], c0, first);
            // a box past the last column reads as zeros
            tma_load_2d(to + 16384, &maps.base, &full[st], c0 + BOX, first);
          }
          if (!none) {
            if constexpr (!TRANS) {
#pragma unroll
              for (int q = 0; q < RT / 64; ++q)
                tma_load_3d(to + S::kBase + q * SLAB * 128, &maps.w, &full[st], q * 64, c0, h.x);
            } else {
#pragma unroll
              for (int q = 0; q < SLAB / 64; ++q)
                tma_load_3d(to + S::kBase + q * RT * 128, &maps.w, &full[st], c0 + q * 64, 0, h.x);
            }
          }
          armed |= 1u << st;
          armed_parity = (armed_parity & ~(1u << st)) | (phase << st);
          if (i == 0 && !none) {
            if (waited)
              ok = load_v(u.tile);
            else
              pending_tile[pending++] = u.tile;
          }
        }
      }
      if (!waited) catch_up();
      if (ok) {
        const int st = step % STAGES;
        const uint32_t phase = (step / STAGES) & 1;
        if (bounded_wait(&empty[st], phase ^ 1, abort_flag, p.status, kTimeout)) {
          meta[st] = kUnitEnd;
          armed &= ~(1u << st);  // its last copy has been read
          for (int i = 0; i < 1 + kCopyWarps; ++i) mbar_arrive(&full[st]);
        }
      }
      // never leave with a copy in flight into this block's shared memory
      for (int s = 0; s < STAGES; ++s)
        if (armed & (1u << s)) mbar_wait(&full[s], (armed_parity >> s) & 1u, kBoundedWaitNs);
      for (int t = a_tiles > S::kABufs ? a_tiles - S::kABufs : 0; t < a_tiles; ++t)
        mbar_wait(&a_full[t % S::kABufs], (t / S::kABufs) & 1, kBoundedWaitNs);
    }
    __syncwarp();
  } else if (warp == 1) {
    // ---------------------------------------------------------- MMA issuer
    if (lane == 0) {
      constexpr uint32_t idesc = idesc_bf16(kTileRows, SLAB) | (TRANS ? kIdescTransB : 0u);
      const int ks = (p.R + 15) / 16;
      int a_tiles = -1, unit = 0;
      for (int step = 0;; ++step) {
        const int st = step % STAGES;
        if (!bounded_wait(&full[st], (step / STAGES) & 1, abort_flag, p.status, kTimeout)) break;
        const int flags = meta[st];
        if (flags & kUnitEnd) break;
        if (flags & kUnitNone) {
          mbar_arrive(&empty[st]);
          continue;
        }
        if (flags & kUnitFirst) {
          ++a_tiles;
          if (!bounded_wait(&a_full[a_tiles % S::kABufs], (a_tiles / S::kABufs) & 1, abort_flag,
                            p.status, kTimeout))
            break;
        }
        const int buf = unit & 1;
        if (!bounded_wait(&acc_empty[buf], ((unit >> 1) & 1) ^ 1, abort_flag, p.status, kTimeout))
          break;
        ++unit;
        tc_fence_after();
        const uint32_t sa = smem_u32(smem + S::kAAt + (a_tiles % S::kABufs) * S::kA);
        const uint32_t sb = smem_u32(smem + st * S::kStage + S::kBase);
#pragma unroll 1
        for (int s = S::kTerms - 1; s >= 0; --s)  // the smallest terms first
#pragma unroll 1
          for (int kk = 0; kk < ks; ++kk)
            mma_bf16_tc(tmem + buf * SLAB,
                        sdesc_kmajor_sw128(sa + (s * (RT / 64) + kk / 4) * 16384 + (kk & 3) * 32),
                        TRANS ? sdesc_mnmajor_sw128(sb + kk * 2048, RT * 128)
                              : sdesc_kmajor_sw128(sb + kk / 4 * (SLAB * 128) + (kk & 3) * 32),
                        idesc, s < S::kTerms - 1 || kk > 0);
        mma_commit(&empty[st]);
        mma_commit(&acc_full[buf]);
        if (flags & kUnitLast) mma_commit(&a_empty[a_tiles % S::kABufs]);
      }
      mma_commit(done);
    }
    __syncwarp();
  } else if (warp < 2 + kExpandWarps) {
    // ------------------------------------------- adding and storing warps
    // thread: row of the tile; warp: a quarter of the rows, half of the slab
    const int quarter = warp & 3, half = (warp - 2) >> 2;
    const int r = quarter * 32 + lane;
    int step = 0, unit = 0, storing = -1;  // storing: stage whose tensor store is under way
    bool ok = true;
    int4 h = make_int4(0, 0, 0, 0);
    int my_row = 0;
    auto read = [&](int tile) {
      const int32_t *rec = u.rec(tile);
      h = *reinterpret_cast<const int4 *>(rec);
      my_row = rec[4 + r];
    };
    if (u.left > 0) read(u.tile);
    while (u.left > 0 && ok) {
      const int bin = h.x, count = h.y, row = my_row;
      const int n = u.here(), slab = u.slab;
      // this warp's rows: how many, and whether one box holds them
      const int mine = count - quarter * 32 < 32 ? count - quarter * 32 : 32;
      const int first = __shfl_sync(~0u, row, 0);
      // rows ascend within a tile
      const bool box = mine == 32 && __shfl_sync(~0u, row, 31) - first == 31;
      u.next_tile();
      if (u.left > 0) read(u.tile);
      const bool none = bin >= p.L;
      if (none && in_place) continue;
      for (int i = 0; i < n; ++i, ++step) {
        const int st = step % STAGES;
        ok = bounded_wait(&full[st], (step / STAGES) & 1, abort_flag, p.status, kTimeout);
        if (!ok) break;
        uint8_t *data = smem + st * S::kStage + half * 16384;
        const int c0 = (slab + i) * SLAB + half * BOX;
        if (!none) {
          const int buf = unit & 1;
          ok = bounded_wait(&acc_full[buf], (unit >> 1) & 1, abort_flag, p.status, kTimeout);
          if (!ok) break;
          ++unit;
          tc_fence_after();
          const uint32_t src =
              tmem + buf * SLAB + half * BOX + (static_cast<uint32_t>(quarter * 32) << 16);
#pragma unroll
          for (int c = 0; c < BOX; c += 32) {
            uint32_t a[32];
            __syncwarp();
            tmem_ld_32x32b_x32(src + c, a);
            tmem_ld_wait();
            if (c + 32 == BOX) {  // the sums are out of tensor memory
              tc_fence_before();
              __syncwarp();
              if (lane == 0) mbar_arrive(&acc_empty[buf]);
            }
#pragma unroll
            for (int q = 0; q < 2 * E; ++q) {  // 16-byte chunks of 32 columns
              uint4 *at = reinterpret_cast<uint4 *>(data + swz128(r, c * E / 16 + q));
              uint4 v = has_base ? *at : make_uint4(0, 0, 0, 0);
              if constexpr (F32) {
                v.x = __float_as_uint(__uint_as_float(v.x) + __uint_as_float(a[q * 4]));
                v.y = __float_as_uint(__uint_as_float(v.y) + __uint_as_float(a[q * 4 + 1]));
                v.z = __float_as_uint(__uint_as_float(v.z) + __uint_as_float(a[q * 4 + 2]));
                v.w = __float_as_uint(__uint_as_float(v.w) + __uint_as_float(a[q * 4 + 3]));
              } else {
                auto add = [&](uint32_t o, int j) {
                  return bf16x2(bf16_lo(o) + __uint_as_float(a[q * 8 + j]),
                                bf16_hi(o) + __uint_as_float(a[q * 8 + j + 1]));
                };
                v = make_uint4(add(v.x, 0), add(v.y, 2), add(v.z, 4), add(v.w, 6));
              }
              *at = v;
            }
          }
        } else if (!has_base) {
#pragma unroll
          for (int q = 0; q < 8; ++q)
            *reinterpret_cast<uint4 *>(data + swz128(r, q)) = make_uint4(0, 0, 0, 0);
        }
        if (storing >= 0 && !box) {  // settle the last tensor store first
          if (lane == 0) {
            bulk_wait_read_all();
            mbar_arrive(&empty[storing]);
          }
          storing = -1;
        }
        if (box) {
          fence_proxy_async_smem();
          __syncwarp();
          if (lane == 0) {
            if (c0 < p.C) tma_store_2d(&maps.out, data + quarter * 4096, c0, first);
            bulk_commit_group();
            if (storing >= 0) {
              bulk_wait_read_but_one();
              mbar_arrive(&empty[storing]);
            }
          }
          storing = st;
        } else {
          __syncwarp();
#pragma unroll
          for (int k = 0; k < 8; ++k) {
            const int rr = k * 4 + (lane >> 3), q = lane & 7;
            const int64_t to = __shfl_sync(~0u, row, rr);
            const int col = c0 + q * (16 / E);
            if (rr < mine && col < p.C &&
                store_ok(p.status, to >= 0 && to < p.M && col + 16 / E <= p.C))
              *reinterpret_cast<uint4 *>(static_cast<uint8_t *>(p.out) +
                                         (to * p.ld_out + col) * E) =
                  *reinterpret_cast<const uint4 *>(data + swz128(quarter * 32 + rr, q));
          }
          // the stage is next written by TMA
          fence_proxy_async_smem();
          __syncwarp();
          if (lane == 0) mbar_arrive(&empty[st]);
        }
      }
    }
    if (lane == 0) {
      bulk_wait_all();  // every tensor store of this warp is complete
      if (storing >= 0) mbar_arrive(&empty[storing]);
    }
    __syncwarp();
  } else {
    // ------------------------------------------------------- copying warps
    // scattered base: 32 rows each, lane: rows 2 i + lane / 16, chunk lane % 16
    const int r0 = (warp - 2 - kExpandWarps) * 32 + (lane >> 4);
    const int q = lane & 15;
    int step = 0;
    bool ok = true;
    LateArrival late;
    for (; u.left > 0 && ok; u.next_tile()) {
      const int32_t *rec = u.rec(u.tile);
      const int4 h = *reinterpret_cast<const int4 *>(rec);
      if (h.x >= p.L && in_place) continue;
      const bool copies = has_base && h.w == 0;
      const int w0 = (warp - 2 - kExpandWarps) * 32, row0 = rec[4 + w0];
      // neighbours (rows ascend within a tile): two boxes
      const bool box = copies && w0 + 32 <= h.y && rec[4 + w0 + 31] - row0 == 31;
      int32_t rows[16];
#pragma unroll
      for (int i = 0; i < 16; ++i) rows[i] = copies ? rec[4 + r0 + 2 * i] : 0;
      const int n = u.here();
      for (int i = 0; i < n; ++i, ++step) {
        const int st = step % STAGES;
        const uint32_t parity = ((step / STAGES) & 1) ^ 1;
        late.before_wait(lane, &empty[st], parity);
        if (lane == 0) ok = bounded_wait(&empty[st], parity, abort_flag, p.status, kTimeout);
        ok = __shfl_sync(~0u, ok, 0);
        if (!ok) break;
        if (!copies || box) {
          late.catch_up(lane);
          if (lane == 0 && box) {
            const int c0 = (u.slab + i) * SLAB;
            uint8_t *to = smem + st * S::kStage + w0 * 128;
            mbar_arrive_expect_tx(&full[st], 8192);
            tma_load_2d(to, &maps.base32, &full[st], c0, row0);
            tma_load_2d(to + 16384, &maps.base32, &full[st], c0 + BOX, row0);
          } else if (lane == 0) {
            mbar_arrive(&full[st]);
          }
          continue;
        }
        const int col = (u.slab + i) * SLAB + q * (16 / E);
        const uint32_t to = smem_u32(smem + st * S::kStage) + (q >> 3) * 16384;
        const uint8_t *src = static_cast<const uint8_t *>(p.base) + static_cast<int64_t>(col) * E;
        if (col < p.C) {
#pragma unroll
          for (int k = 0; k < 16; ++k) {
            if (r0 - (lane >> 4) + 2 * k >= h.y) break;
            if (r0 + 2 * k < h.y)
              cp_async16(to + swz128(r0 + 2 * k, q & 7), src + rows[k] * p.ld_base * E, true);
          }
        }
        cp_async_commit();
        late.push(lane, &full[st]);
      }
    }
    late.catch_up(lane);
    cp_async_wait<0>();
  }
  bounded_wait(done, 0, abort_flag, p.status, kTimeout);

  tc_fence_before();
  __syncthreads();
  if (warp == 1) {
    __syncwarp();
    tc_fence_after();
    tmem_dealloc(tmem, 2 * SLAB);
  }
}

// ---------------------------------------------------------------------- outer
// out[a](c, j) = f sum_{m of a} src[m][c] v[m][j]: dB[a][n][j] (src dy, v t, f =
// scale) and dA[a][j][k] (src x, v dt, f = 1, stored transposed).  A cluster
// takes a slab of 128 columns c; its blocks take equal shares of the row tiles
// of all adapters in order, 64 rows a stage: src's rows as a TMA box where 64
// neighbours are the adapter's (else boxes of 32, or copies by a warp) and v's
// box; both are operands whose rows run along the contraction, M = 128 columns of
// src by N = RT, sums in tensor memory, one buffer in use and one being stored.
// Past a tile's last row both are zero.
// An adapter whose tiles lie in one block goes straight to memory.  A block
// shares at most its first and its last adapter with its neighbours: those
// partial sums meet in distributed shared memory, added in block order.
// Bound by the rows' way from HBM: 8858 rows of two adapters, 6144 + 1536 columns,
// rank 64, 138 MB in 46 us from a cold L2 (profiler; 256 bytes a row and stage).
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
  int32_t beside;  // the kernel ahead is the expansion, not the contraction
  const int32_t *plan;
  int64_t M;
  int32_t R, L;
  int *status;
};
struct OuterMaps {
  CUtensorMap src[2], src32[2], v[2];  // rows of a box: 64, 32, 64
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
  const CUtensorMap *tm_src32 = second ? &maps.src32[1] : &maps.src32[0];
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
  // Behind the expansion: that one lets this kernel begin when the contraction
  // is complete, and nothing here touches what it writes, so the two run side by
  // side, on the SMs that the expansion leaves free or has left (a block of each
  // needs more shared memory than an SM has); the wait at the end keeps the stream's
  // order for what comes next.
  if (!p.beside) grid_dependency_wait();

  const int cols = sd.C - c0 < kOuterSlab ? sd.C - c0 : kOuterSlab;
  const int64_t grads = static_cast<int64_t>(p.L) * p.R * sd.C;  // elements of sd.out
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
      late.before_wait(lane, &empty[st], phase ^ 1);
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
      const int halves = (h.y + kOuterRows - 1) / kOuterRows;
      const bool head = h.x != bin_before;
      const bool tail = tile + 1 == t_hi || next.h.x != h.x;
      for (int q = 0; q < halves && ok; ++q) {
        // The stage's two groups of 32 rows, a row a lane: neighbours (rows ascend
        // within a tile) come as boxes of 64 or 32 rows, others by copies.
        const int group[2] = {q == 0 ? now.rows[0] : now.rows[2],
                              q == 0 ? now.rows[1] : now.rows[3]};
        int at[2];
        bool boxes[2];
#pragma unroll
        for (int j = 0; j < 2; ++j) {
          at[j] = __shfl_sync(~0u, group[j], 0);
          boxes[j] = h.y - q * kOuterRows >= 32 * (j + 1) &&
                     __shfl_sync(~0u, group[j], 31) - at[j] == 31;
        }
        const bool box = boxes[0] && boxes[1] && at[1] - at[0] == 32;
        const int n_boxes = boxes[0] + boxes[1];
        const int st = take((head && q == 0 ? kStageFirst : 0) |
                                (tail && q == halves - 1 ? kStageLast : 0),
                            S::kV + n_boxes * (wide ? 2 : 1) * 4096);
        if (!ok) break;
        uint8_t *src = smem + st * S::kStage;
        if (lane == 0) {
          if (box) {
            tma_load_2d(src, tm_src, &full[st], c0, at[0]);
            if (wide) tma_load_2d(src + 8192, tm_src, &full[st], c0 + 64, at[0]);
          } else {
#pragma unroll
            for (int j = 0; j < 2; ++j)
              if (boxes[j]) {
                tma_load_2d(src + j * 4096, tm_src32, &full[st], c0, at[j]);
                if (wide) tma_load_2d(src + 8192 + j * 4096, tm_src32, &full[st], c0 + 64, at[j]);
              }
          }
#pragma unroll
          for (int s = 0; s < TERMS; ++s)
#pragma unroll
            for (int b = 0; b < RT / 64; ++b)
              tma_load_3d(src + S::kSrc + (s * (RT / 64) + b) * 8192, tm_v, &full[st], b * 64,
                          tile * kTileRows + q * kOuterRows, s);
        }
        if (n_boxes == 2) {
          late.catch_up(lane);
          if (lane == 0) mbar_arrive(&full[st]);
        } else {
          const int c = lane & 15, col = c0 + c * 8;
          const uint32_t to = smem_u32(src) + (c >> 3) * 8192;
          const bool in_cols = col < sd.C;
#pragma unroll
          for (int j = 0; j < 2; ++j) {
            if (boxes[j]) continue;
            int32_t rows[16];  // all exchanged before the first copy
#pragma unroll
            for (int i = 0; i < 16; ++i)
              rows[i] = __shfl_sync(~0u, group[j], i * 2 + (lane >> 4));
            if (c < 8 || wide) {
#pragma unroll
              for (int i = 0; i < 16; ++i) {
                // zeros past the tile's last row, which meet zeros of v
                const int r = j * 32 + i * 2 + (lane >> 4);
                const bool in = in_cols && q * kOuterRows + r < h.y;
                cp_async16(to + swz128(r, c & 7), sd.src + rows[i] * sd.ld + (in ? col : 0), in);
              }
            }
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
          const int js = p.R - j0 < 32 ? p.R - j0 : 32;  // of this thread's stores
          const int64_t end = sd.transposed
                                  ? obase + static_cast<int64_t>(j0 + js - 1) * sd.C + c0 + c + 1
                                  : obase + static_cast<int64_t>(c0 + c) * p.R + j0 + js;
          if (c < cols && js > 0 && store_ok(p.status, end <= grads)) {
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
          const int64_t end = sd.transposed
                                  ? obase + static_cast<int64_t>(j + 3) * sd.C + c0 + c + 1
                                  : obase + static_cast<int64_t>(c0 + c) * p.R + j + 4;
          if (!store_ok(p.status, end <= grads)) continue;
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
        if (store_ok(p.status, at < grads))
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
  if (p.beside) grid_dependency_wait();
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

// Tensor map of [d2][d1][d0] with row stride ld (elements), boxes of 128 bytes by
// `rows`, 128-byte swizzle; d2 == 0: two dimensions.
cudaError_t tile_map(CUtensorMap *map, bool f32, const void *ptr, int64_t d0, int64_t d1,
                     int64_t d2, int64_t ld, int rows) {
  EncodeTiledFn enc = tensor_map_encoder();
  if (enc == nullptr) return cudaErrorNotSupported;
  const int elem = f32 ? 4 : 2;
  if (d1 <= 1) ld = (d0 + 7) / 8 * 8;  // one row: its stride may be anything
  const cuuint64_t dims[3] = {static_cast<cuuint64_t>(d0), static_cast<cuuint64_t>(d1),
                              static_cast<cuuint64_t>(d2)};
  const cuuint64_t strides[2] = {static_cast<cuuint64_t>(ld) * elem,
                                 static_cast<cuuint64_t>(ld) * elem * static_cast<cuuint64_t>(d1)};
  const cuuint32_t box[3] = {static_cast<cuuint32_t>(128 / elem), static_cast<cuuint32_t>(rows), 1};
  const cuuint32_t estr[3] = {1, 1, 1};
  return enc(map, f32 ? CU_TENSOR_MAP_DATA_TYPE_FLOAT32 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16,
             d2 == 0 ? 2 : 3, const_cast<void *>(ptr), dims, strides, box, estr,
             CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
             CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
             CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS
             ? cudaSuccess
             : cudaErrorInvalidValue;
}
cudaError_t bf16_map(CUtensorMap *map, const void *ptr, int64_t d0, int64_t d1, int64_t d2,
                     int64_t ld, int rows) {
  return tile_map(map, false, ptr, d0, d1, d2, ld, rows);
}

template <int RT, bool TRANS, int TERMS>
cudaError_t run_contract(const uint16_t *w, const ContractArgs &a, cudaStream_t stream) {
  CUtensorMap tm_in, tm_in32, tm_w;
  cudaError_t e = bf16_map(&tm_in, a.in, a.C, a.M, 0, a.ld, kTileRows);
  if (e == cudaSuccess) e = bf16_map(&tm_in32, a.in, a.C, a.M, 0, a.ld, 32);
  if (e == cudaSuccess)
    e = TRANS ? bf16_map(&tm_w, w, a.R, a.C, a.L, a.R, 64)
              : bf16_map(&tm_w, w, a.C, a.R, a.L, a.C, RT);
  if (e != cudaSuccess) return e;
  // Slices of the contracted dimension: as many as let all tiles run at once
  // (two blocks per SM), none shorter than 128 columns.
  int slices = 1;
  while (slices < 8 && a.C >= 128 * slices * 2 && a.max_tiles * slices * 2 <= 2 * sm_count())
    slices *= 2;
  return launch<lora_contract_kernel<RT, TRANS, TERMS>>(
      dim3(static_cast<unsigned>(a.max_tiles), slices), kContractThreads,
      ContractSmem<RT>::kBytes, slices, 1, stream, tm_in, tm_in32, tm_w, a);
}

template <int RT, bool TRANS, bool F32, int TERMS>
cudaError_t run_expand(const uint16_t *w, const uint16_t *v, const ExpandArgs &a,
                       cudaStream_t stream) {
  using S = ExpandSmem<RT, F32, TERMS>;
  ExpandMaps maps;
  const void *base = a.base ? a.base : a.out;  // not read without a base
  cudaError_t e = tile_map(&maps.base, F32, base, a.C, a.M, 0, a.base ? a.ld_base : a.ld_out,
                           kTileRows);
  if (e == cudaSuccess)
    e = tile_map(&maps.base32, F32, base, a.C, a.M, 0, a.base ? a.ld_base : a.ld_out, 32);
  if (e == cudaSuccess) e = tile_map(&maps.out, F32, a.out, a.C, a.M, 0, a.ld_out, 32);
  if (e == cudaSuccess)
    e = TRANS ? bf16_map(&maps.w, w, a.C, a.R, a.L, a.C, RT)
              : bf16_map(&maps.w, w, a.R, a.C, a.L, a.R, S::kSlab);
  if (e == cudaSuccess)
    e = bf16_map(&maps.v, v, a.R, a.max_tiles * kTileRows, S::kTerms, a.R, kTileRows);
  if (e != cudaSuccess) return e;
  const int64_t units = a.max_tiles * ((a.C + S::kSlab - 1) / S::kSlab);
  const int sms = sm_count();
  return launch<lora_expand_kernel<RT, TRANS, F32, TERMS>>(
      dim3(static_cast<unsigned>(units < sms ? units : sms)), kExpandThreads, S::kBytes, 1, 0,
      stream, maps, a);
}

template <int RT, int TERMS>
cudaError_t run_outer(const OuterMaps &maps, const OuterArgs &a, cudaStream_t stream) {
  using S = OuterSmem<RT, TERMS>;
  const int slabs = a.slabs0 + (a.side[1].C + kOuterSlab - 1) / kOuterSlab;
  // Blocks of a slab: as many (up to the portable cluster size, with 64 rows each
  // at least) as let all slabs run at once.  A cluster lies within one
  // of the GPU's partitions, which leaves some places empty: 60 slabs by 4 take
  // 42 us, by 7 (three blocks per SM) two rounds and 80 us.
  int shares = 1;
  for (int n = 2; n <= 8 && a.M >= kTileRows / 2 * n; ++n)
    if (static_cast<int64_t>(slabs) * n * 16 <= static_cast<int64_t>(S::kPerSm) * sm_count() * 15)
      shares = n;
  return launch<lora_outer_kernel<RT, TERMS>>(dim3(slabs * shares), kOuterThreads, S::kBytes,
                                              shares, 0, stream, maps, a);
}

// The kernel for few rows: up to a pass of it (16 rows) or, where these can belong
// to several adapters, two, and a second product that eight blocks do quickly.
// 1536 -> 1536, rank 16, in place: 5.6 us for one row, 6.2 for 16 rows of 8
// adapters or of one, 10.9 for 32 rows of one, against 9.9, 13.0, 9.9 and 9.9 by
// tiles; rank 128: 8.3, 9.3, 10.6, 19.7 against 11.1, 14.2, 11.5, 11.5.  1536 ->
// 6144, rank 64, one row: 13.1 against 10.3.
bool few_rows(const LoraRequest &q) {
  return q.M <= (q.L > 1 ? 2 : 1) * kFewRows && q.N * q.R <= 1 << 18;
}

// Ranks are padded to 64 (128) columns: the boxes' columns past R read as zero.
template <typename F>
cudaError_t by_rank(int R, F &&f) {
  if (R <= 64) return f(std::integral_constant<int, 64>());
  return f(std::integral_constant<int, 128>());
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
  const ContractArgs c = {q.dy, q.lddy, q.scale, q.plan, q.t, vdt, vt,
                          q.M, max_tiles, N, q.R, q.L, q.status};
  cudaError_t e = by_rank(q.R, [&](auto rt) {
    return run_contract<decltype(rt)::value, true, TERMS>(q.B, c, stream);
  });
  if (e == cudaSuccess && q.dx != nullptr) {
    const ExpandArgs x = {q.plan, q.base, q.ld_base, q.dx, q.lddx, q.M,
                          max_tiles, K, q.R, q.L, q.status};
    // dt's only term, or the first two of three (16 bits: they are cut off, not
    // rounded)
    e = by_rank(q.R, [&](auto rt) {
      return run_expand<decltype(rt)::value, true, false, TERMS == 1 ? 1 : 2>(q.A, vdt, x, stream);
    });
  }
  if (e == cudaSuccess && q.dA != nullptr) {
    OuterMaps maps;
    OuterArgs o = {};
    o.side[0] = {q.dy, q.lddy, q.scale, q.dB, N, 0};
    o.side[1] = {q.x, q.ldx, nullptr, q.dA, K, 1};
    o.slabs0 = (N + kOuterSlab - 1) / kOuterSlab;
    o.beside = q.dx != nullptr;
    o.plan = q.plan;
    o.M = q.M;
    o.R = q.R;
    o.L = q.L;
    o.status = q.status;
    e = bf16_map(&maps.src[0], q.dy, N, q.M, 0, q.lddy, kOuterRows);
    if (e == cudaSuccess) e = bf16_map(&maps.src[1], q.x, K, q.M, 0, q.ldx, kOuterRows);
    if (e == cudaSuccess) e = bf16_map(&maps.src32[0], q.dy, N, q.M, 0, q.lddy, 32);
    if (e == cudaSuccess) e = bf16_map(&maps.src32[1], q.x, K, q.M, 0, q.ldx, 32);
    if (e == cudaSuccess) e = bf16_map(&maps.v[0], vt, q.R, rows, TERMS, q.R, kOuterRows);
    if (e == cudaSuccess) e = bf16_map(&maps.v[1], vdt, q.R, rows, TERMS, q.R, kOuterRows);
    if (e == cudaSuccess)
      e = by_rank(q.R, [&](auto rt) {
        return run_outer<decltype(rt)::value, TERMS>(maps, o, stream);
      });
  }
  return e;
}

template <bool F32>
cudaError_t run_few(const LoraRequest &q, cudaStream_t stream) {
  const FewArgs a = {q.x, q.A, q.B, q.scale, q.plan, q.base, q.y, q.t, q.ldx, q.ld_base, q.ldy, q.M,
                     static_cast<int32_t>(q.N), static_cast<int32_t>(q.K), q.R, q.L, q.status};
  return by_rank(q.R, [&](auto rt) {
    constexpr int RT = decltype(rt)::value;
    return launch<lora_few_kernel<RT, F32>>(
        dim3(static_cast<unsigned>(plan_max_tiles(q.M, q.L)), kFewCluster), kFewThreads,
        FewSmem<RT, F32 ? 3 : 1>::kBytes, kFewCluster, 1, stream, a);
  });
}

template <bool F32>
cudaError_t run_forward(const LoraRequest &q, cudaStream_t stream) {
  if (few_rows(q)) return run_few<F32>(q, stream);
  const int64_t max_tiles = plan_max_tiles(q.M, q.L);
  uint16_t *v = static_cast<uint16_t *>(q.workspace);
  const ContractArgs c = {q.x, q.ldx, q.scale, q.plan, q.t, v, nullptr, q.M,
                          max_tiles, static_cast<int32_t>(q.K), q.R, q.L, q.status};
  const ExpandArgs x = {q.plan, q.base, q.ld_base, q.y, q.ldy, q.M,
                        max_tiles, static_cast<int32_t>(q.N), q.R, q.L, q.status};
  return by_rank(q.R, [&](auto rt) {
    constexpr int RT = decltype(rt)::value;
    const cudaError_t e = run_contract<RT, false, F32 ? 3 : 1>(q.A, c, stream);
    return e != cudaSuccess ? e : run_expand<RT, false, F32, F32 ? 3 : 1>(q.B, v, x, stream);
  });
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
  // the limit for any L: calls of two threads must not lower each other's
  const int bytes = (kPlanWarps * (L + 1) + 2 * (L + 2)) * 4;
  const cudaError_t e = allow_smem<lora_plan_kernel>((kPlanWarps * 1025 + 2 * 1026) * 4);
  if (e != cudaSuccess) return e;
  lora_plan_kernel<<<1, kPlanWarps * 32, bytes, stream>>>(adapter, static_cast<int32_t>(M), L,
                                                          plan, status);
  return cudaGetLastError();
}

cudaError_t launch_lora_forward(const LoraRequest &q, cudaStream_t stream) {
  return q.f32 ? run_forward<true>(q, stream) : run_forward<false>(q, stream);
}

cudaError_t launch_lora_backward(const LoraRequest &q, cudaStream_t stream) {
  return q.f32 ? run_backward<3>(q, stream) : run_backward<1>(q, stream);
}

}  // namespace sq
