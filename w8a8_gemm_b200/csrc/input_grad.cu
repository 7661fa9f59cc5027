// input_grad.cu -- the gradient of a frozen quantized linear with respect to
// its input, straight through the activation quantizer:
//   dx[m][k] = sum_n dy[m][n] W~[n][k],  W~[n][k] = s_w[i(k)][n] W^[n][k] / d[g(n)][k].
//
// Two kernels.  The first writes W~, rounded to bf16, into the caller's
// workspace (3 N K bytes of traffic, a few percent of the product): steps and
// divisors vary along both dimensions, so they belong to the weight.  The
// rounding to bf16 is one more rounding of the size of dy's own and averages
// over the N terms.
//
// The second is a bf16 product on the tensor cores: persistent pairs of blocks,
// each pair 256 x BN output tiles of one tcgen05.mma kind::f16, cta_group::2.
// A block fetches 128 rows of dy and BN / 2 columns of W~ a step (64 terms of
// the contraction) by TMA into a ring of stages, 128-byte swizzled; W~ lies
// contiguous along the output, an MN-major operand.  The sums are fp32 in tensor
// memory, in two buffers, so that a tile's epilogue runs under the next tile's
// products.  Where there are few tiles, several pairs of a cluster share one's
// contraction and add their sums in a fixed order.  What bounds it is the way of
// the operands from L2 to an SM, 40 to 60 bytes a clock: one block by itself with
// 128 x 256 tiles fetches 48 KB for 512 clocks of products, a pair 32 KB a block.
// 8858 x 6144 -> 1536: 121 to 126 us in a replayed graph on one input (129 with one
// block a tile), 142 to 146 a call with new ones, under the power cap; the product
// by itself 120 us at 1.58 GHz (profiler: 1389 TFLOP/s, tensor pipe 73%).  1109 x 1536
// -> 1536: 18.9 us, 19.3 a call.
#include <cooperative_groups.h>
#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_fp8.h>
#include <cuda_runtime.h>
#include <math.h>
#include <stdint.h>

#include "bf16.cuh"
#include "input_grad_plan.h"
#include "sq_internal.h"

namespace cg = cooperative_groups;

namespace sq {
namespace {

// ------------------------------------------------------------------------- W~
// w [N][K].  A thread has 8 neighbouring channels of kDeqRows rows of the weight,
// all loads under way at once; a block 256 channels of 32 rows.  A channel's divisor
// is inverted once (one rounding more; with a division for every code 1536 x
// 1536 took 7.6 us for 6.7), unless its inverse is past the largest number.
constexpr int kDeqThreads = 256, kDeqLanes = kDeqThreads / 32, kDeqRows = 4;
__global__ void __launch_bounds__(kDeqThreads) dequant_kernel(
    const int8_t *__restrict__ wq, const float *__restrict__ s_w, const float *__restrict__ d,
    int64_t N, int64_t K, const __grid_constant__ SegParams seg, uint16_t *__restrict__ w,
    int *status) {
  grid_dependency_wait();
  grid_dependency_launch();
  const int64_t k = (static_cast<int64_t>(blockIdx.x) * 32 + (threadIdx.x & 31)) * 8;
  if (k >= K) return;  // K % 16 == 0
  const int64_t n0 = static_cast<int64_t>(blockIdx.y) * kDeqLanes * kDeqRows + (threadIdx.x >> 5);
  // input segments are at least 32 wide and aligned to 32: one for 8 codes
  const int i = seg.S > 1 ? seg_index(seg.off, seg.n_seg, k) : 0;
  uint2 v[kDeqRows];
  float s[kDeqRows];
  float inv[8], dv[8];  // of activation group `group`
  bool inverts = true;
  int group = -1;
  auto divisors = [&](int64_t n) {
    const int g = seg.G > 1 ? seg_index(seg.off, seg.n_seg, n) : 0;
    if (g == group) return;
    group = g;
    inverts = true;
#pragma unroll
    for (int j = 0; j < 8; ++j) dv[j] = d[g * K + k + j];
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      inv[j] = __frcp_rn(dv[j]);
      inverts = inverts && fabsf(inv[j]) < INFINITY;
    }
  };
#pragma unroll
  for (int r = 0; r < kDeqRows; ++r) {
    const int64_t n = n0 + r * kDeqLanes;
    if (n < N) {
      v[r] = *reinterpret_cast<const uint2 *>(wq + n * K + k);
      s[r] = s_w[i * N + n] * (seg.w4 ? 0.0625f : 1.0f);  // W4 operands hold 16 q
    }
  }
#pragma unroll
  for (int r = 0; r < kDeqRows; ++r) {
    const int64_t n = n0 + r * kDeqLanes;
    if (n >= N) break;
    float q[8];
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      const uint32_t byte = ((j < 4 ? v[r].x : v[r].y) >> ((j & 3) * 8)) & 0xFFu;
      if (seg.fp8) {
        const __half_raw h = __nv_cvt_fp8_to_halfraw(static_cast<__nv_fp8_storage_t>(byte),
                                                     __NV_E4M3);
        q[j] = __half2float(__half(h));
      } else {
        q[j] = static_cast<float>(static_cast<int8_t>(byte));
      }
      q[j] *= s[r];
    }
    if (d != nullptr) {
      divisors(n);
#pragma unroll
      for (int j = 0; j < 8; ++j) q[j] = inverts ? q[j] * inv[j] : __fdiv_rn(q[j], dv[j]);
    }
    if (store_ok(status, n * K + k + 8 <= N * K))
      *reinterpret_cast<uint4 *>(w + n * K + k) = make_uint4(
          bf16x2(q[0], q[1]), bf16x2(q[2], q[3]), bf16x2(q[4], q[5]), bf16x2(q[6], q[7]));
  }
}

// -------------------------------------------------------------------- product
constexpr int BM = kGradTileRows / 2, BK = kGradStep;  // rows of a block, terms of a step
constexpr int kEpiWarps = 8;
constexpr int kGemmThreads = 64 + 32 * kEpiWarps;

template <int BN>
struct GemmSmem {
  static constexpr int A = BM * BK * 2, B = BN / 2 * BK * 2;
  static constexpr int STAGE = A + B;
  static constexpr int STAGES = BN == 256 ? 6 : 8;
  static constexpr int BARS = STAGES * STAGE;
  static constexpr int BYTES = BARS + (2 * STAGES + 5) * 8 + 16 + 1024;
};

struct GradArgs {
  int32_t M, K;         // output rows and columns
  int32_t num_n_tiles, num_tiles, num_kb;
  int32_t splits;       // pairs that share a tile's contraction; above 1 a cluster has one tile
  uint16_t *dx;
  int64_t lddx;
  int *status;
};

__device__ __forceinline__ bool wait_bar(uint64_t *bar, uint32_t parity, volatile int *abort_flag,
                                         int *status) {
  return bounded_wait(bar, parity, abort_flag, status, SQ_ERR_DEVICE_TIMEOUT);
}

// Barriers: `full` (both blocks' copies) and `acc_empty` (both blocks' epilogues)
// count in the even block, which issues the products; `empty` and `acc_full`
// are committed to in both.
template <int BN>
__global__ void __launch_bounds__(kGemmThreads, 1)
    input_grad_kernel(const __grid_constant__ CUtensorMap tmA,
                      const __grid_constant__ CUtensorMap tmB, const GradArgs p) {
  using L = GemmSmem<BN>;
  constexpr int STAGES = L::STAGES;
  constexpr int COLS = 2 * BN;  // two accumulator buffers
  constexpr int kPartRow = BN + 4;  // floats
  static_assert(BM * kPartRow * 4 <= L::BARS, "partial sums reuse the stages");
  extern __shared__ uint8_t smem_raw[];
  // the same offset in both blocks: the window starts at the same address
  uint8_t *smem = reinterpret_cast<uint8_t *>(
      (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~static_cast<uintptr_t>(1023));
  uint64_t *full = reinterpret_cast<uint64_t *>(smem + L::BARS);
  uint64_t *empty = full + STAGES;
  uint64_t *acc_full = empty + STAGES;
  uint64_t *acc_empty = acc_full + 2;
  uint64_t *mma_done = acc_empty + 2;
  uint32_t *tmem_slot = reinterpret_cast<uint32_t *>(mma_done + 1);
  volatile int *abort_flag = reinterpret_cast<volatile int *>(tmem_slot + 1);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  cg::cluster_group cluster = cg::this_cluster();
  // A cluster has one pair, or the pairs that share a tile's contraction.
  const uint32_t even = cluster.block_rank() & ~1u, rank = cluster.block_rank() & 1u;
  const uint32_t both = 3u << even;
  const int pair = static_cast<int>(even >> 1);
  const int first = blockIdx.x / (2 * p.splits), step = gridDim.x / (2 * p.splits);
  const int kb_lo = p.num_kb * pair / p.splits;
  const int steps = p.num_kb * (pair + 1) / p.splits - kb_lo;  // of 64 terms

  if (threadIdx.x == 0) {
    for (int s = 0; s < STAGES; ++s) {
      mbar_init(&full[s], 1);
      mbar_init(&empty[s], 1);
    }
    for (int b = 0; b < 2; ++b) {
      mbar_init(&acc_full[b], 1);
      mbar_init(&acc_empty[b], 2 * kEpiWarps);
    }
    mbar_init(mma_done, 1);
    *abort_flag = 0;
    fence_mbar_init();
    prefetch_tmap(&tmA);
    prefetch_tmap(&tmB);
  }
  if (warp == 1) {
    tmem_alloc_pair(tmem_slot, COLS);
    tmem_relinquish_pair();
  }
  __syncwarp();
  tc_fence_before();
  cluster.sync();  // both blocks' barriers and columns stand
  tc_fence_after();
  const uint32_t tmem_base = *tmem_slot;
  // dy was complete before the kernel ahead of this one began; only W~, which that
  // one writes, has to be waited for
  if (warp != 0) grid_dependency_wait();

  if (warp == 0) {
    if (lane == 0) {
      int stage = 0, early = 0;
      uint32_t phase = 0, armed = 0, armed_parity = 0;
      bool gave_up = false;
      // the first tile's rows of dy, as many stages as there are
      if (first < p.num_tiles) {
        early = steps < STAGES ? steps : STAGES;
        for (int i = 0; i < early; ++i) {
          if (rank == 0) mbar_arrive_expect_tx(&full[i], 2 * L::STAGE);
          tma_load_2d_pair(smem + i * L::STAGE, &tmA, cluster_addr(&full[i], even),
                           (kb_lo + i) * BK, (first / p.num_n_tiles * 2 + rank) * BM);
        }
      }
      grid_dependency_wait();
      for (int tile = first; tile < p.num_tiles; tile += step) {
        const int row = (tile / p.num_n_tiles * 2 + rank) * BM;
        const int col = tile % p.num_n_tiles * BN + rank * (BN / 2);
        for (int i = 0; i < steps; ++i) {
          const int kb = kb_lo + i;
          if (!wait_bar(&empty[stage], phase ^ 1, abort_flag, p.status)) {
            gave_up = true;
            goto producer_done;
          }
          uint8_t *sa = smem + stage * L::STAGE;
          const uint32_t bar = cluster_addr(&full[stage], even);
          if (tile != first || i >= early) {
            if (rank == 0) mbar_arrive_expect_tx(&full[stage], 2 * L::STAGE);
            tma_load_2d_pair(sa, &tmA, bar, kb * BK, row);
          }
#pragma unroll
          for (int b = 0; b < BN / 128; ++b)
            tma_load_2d_pair(sa + L::A + b * 8192, &tmB, bar, col + b * 64, kb * BK);
          armed |= 1u << stage;
          armed_parity = (armed_parity & ~(1u << stage)) | (phase << stage);
          if (++stage == STAGES) {
            stage = 0;
            phase ^= 1;
          }
        }
      }
    producer_done:
      // Never leave with a copy, or a product's arrival, under way into this
      // block's shared memory.  After a wait that ran out, the even block's
      // barriers tell of the copies of both; the odd block gives its own, which
      // have had that wait's seconds, a little more.
      for (int s = 0; s < STAGES; ++s) {
        const uint32_t parity = (armed_parity >> s) & 1u;
        if (!(armed & (1u << s))) continue;
        if (!gave_up && wait_bar(&empty[s], parity, abort_flag, p.status)) continue;
        gave_up = true;
        if (rank == 0) mbar_wait(&full[s], parity, kBoundedWaitNs);
      }
      if (gave_up && rank == 1) {
        const uint64_t t0 = globaltimer_ns();
        while (globaltimer_ns() - t0 < kBoundedWaitNs / 1000) {
        }
      }
    }
  } else if (warp == 1) {
    if (lane == 0 && rank == 0) {
      constexpr uint32_t idesc = idesc_bf16(2 * BM, BN) | kIdescTransB;
      int stage = 0;
      uint32_t phase = 0, iter = 0;
      for (int tile = first; tile < p.num_tiles; tile += step, ++iter) {
        const uint32_t buf = iter & 1;
        if (!wait_bar(&acc_empty[buf], ((iter >> 1) & 1) ^ 1, abort_flag, p.status))
          goto mma_exit;
        fence_cluster();  // the other block's reads of this buffer come before
        tc_fence_after();
        const uint32_t acc = tmem_base + buf * BN;
        for (int i = 0; i < steps; ++i) {
          if (!wait_bar(&full[stage], phase, abort_flag, p.status)) goto mma_exit;
          tc_fence_after();
          const uint32_t sa = smem_u32(smem + stage * L::STAGE), sb = sa + L::A;
#pragma unroll
          for (int kk = 0; kk < BK / 16; ++kk)
            mma_bf16_pair(acc, sdesc_kmajor_sw128(sa + kk * 32),
                          sdesc_mnmajor_sw128(sb + kk * 2048, 8192), idesc, (i | kk) != 0);
          mma_commit_pair(&empty[stage], both);
          if (++stage == STAGES) {
            stage = 0;
            phase ^= 1;
          }
        }
        mma_commit_pair(&acc_full[buf], both);
      }
    mma_exit:
      mma_commit_pair_here(mma_done);
      mbar_wait(mma_done, 0, kBoundedWaitNs);
    }
  } else {
    const int quarter = warp & 3;         // TMEM lanes this warp may read
    const int half = (warp - 2) >> 2;     // which half of the columns
    uint32_t iter = 0;
    for (int tile = first; tile < p.num_tiles; tile += step, ++iter) {
      const uint32_t buf = iter & 1;
      if (!wait_bar(&acc_full[buf], (iter >> 1) & 1, abort_flag, p.status)) break;
      tc_fence_after();
      const int row = (tile / p.num_n_tiles * 2 + rank) * BM + quarter * 32 + lane;
      const int nt = tile % p.num_n_tiles;
      const uint32_t src = tmem_base + buf * BN + (static_cast<uint32_t>(quarter * 32) << 16);
#pragma unroll 1
      for (int c = half * (BN / 2); c < (half + 1) * (BN / 2); c += 32) {
        uint32_t r[32];
        __syncwarp();
        tmem_ld_32x32b_x32(src + c, r);
        tmem_ld_wait();
        const int col = nt * BN + c;
        if (p.splits > 1) {  // this pair's sums: in the stages, all of which have been used
          float *to = reinterpret_cast<float *>(smem) + (quarter * 32 + lane) * kPartRow + c;
#pragma unroll
          for (int j = 0; j < 32; j += 4)
            *reinterpret_cast<uint4 *>(to + j) = make_uint4(r[j], r[j + 1], r[j + 2], r[j + 3]);
          continue;
        }
#pragma unroll
        for (int q = 0; q < 4; ++q) {  // K % 16 == 0: 8 columns are all in or all out
          const int c8 = col + q * 8;
          if (row < p.M && c8 < p.K && store_ok(p.status, c8 + 8 <= p.K)) {
            uint32_t o[4];
#pragma unroll
            for (int j = 0; j < 4; ++j)
              o[j] = bf16x2(__uint_as_float(r[q * 8 + 2 * j]),
                            __uint_as_float(r[q * 8 + 2 * j + 1]));
            *reinterpret_cast<uint4 *>(p.dx + static_cast<int64_t>(row) * p.lddx + c8) =
                make_uint4(o[0], o[1], o[2], o[3]);
          }
        }
      }
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive_cluster(cluster_addr(&acc_empty[buf], even));
    }
  }

  __syncwarp();
  tc_fence_before();
  cluster.sync();  // no products and no arrivals under way in any block
  if (p.splits > 1) {
    // The pairs' sums of the tile, added in their order: a block a share of its rows.
    const int rows = BM / p.splits, nt = first % p.num_n_tiles;
    for (int e = threadIdx.x; e < rows * (BN / 8); e += kGemmThreads) {
      const int m = pair * rows + e / (BN / 8), c = e % (BN / 8) * 8;
      float v[8] = {0.0f, 0.0f, 0.0f, 0.0f, 0.0f, 0.0f, 0.0f, 0.0f};
      for (int q = 0; q < p.splits; ++q) {
        const float4 *src = reinterpret_cast<const float4 *>(
            cluster.map_shared_rank(reinterpret_cast<float *>(smem), 2 * q + rank) +
            m * kPartRow + c);
        const float4 a = src[0], b = src[1];
        v[0] += a.x, v[1] += a.y, v[2] += a.z, v[3] += a.w;
        v[4] += b.x, v[5] += b.y, v[6] += b.z, v[7] += b.w;
      }
      const int row = (first / p.num_n_tiles * 2 + rank) * BM + m, c8 = nt * BN + c;
      if (row < p.M && c8 < p.K && store_ok(p.status, c8 + 8 <= p.K))
        *reinterpret_cast<uint4 *>(p.dx + static_cast<int64_t>(row) * p.lddx + c8) =
            make_uint4(bf16x2(v[0], v[1]), bf16x2(v[2], v[3]), bf16x2(v[4], v[5]),
                       bf16x2(v[6], v[7]));
    }
    cluster.sync();  // no block leaves while its sums are read
  }
  if (warp == 1) {
    __syncwarp();
    tc_fence_after();
    tmem_dealloc_pair(tmem_base, COLS);
  }
}

sq_status tensor_map_2d(CUtensorMap *map, const void *ptr, int64_t inner, int64_t outer,
                        int64_t ld, int box_rows) {
  EncodeTiledFn enc = tensor_map_encoder();
  if (enc == nullptr) return SQ_ERR_CUDA;
  if (outer <= 1) ld = (inner + 7) / 8 * 8;  // one row: its stride may be anything
  const cuuint64_t dims[2] = {static_cast<cuuint64_t>(inner), static_cast<cuuint64_t>(outer)};
  const cuuint64_t strides[1] = {static_cast<cuuint64_t>(ld) * 2};
  const cuuint32_t box[2] = {BK, static_cast<cuuint32_t>(box_rows)};
  const cuuint32_t estr[2] = {1, 1};
  return enc(map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 2, const_cast<void *>(ptr), dims, strides, box,
             estr, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
             CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
             CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS
             ? SQ_OK
             : SQ_ERR_CUDA;
}

template <int BN>
sq_status run_gemm(const InputGradRequest &r, const uint16_t *w, const InputGradPlan &plan,
                   cudaStream_t stream) {
  using L = GemmSmem<BN>;
  static_assert(L::BYTES <= 232448, "dynamic shared memory above the per-block limit");
  CUtensorMap tmA, tmB;
  sq_status st = tensor_map_2d(&tmA, r.dy, r.N, r.M, r.lddy, BM);
  if (st == SQ_OK) st = tensor_map_2d(&tmB, w, r.K, r.N, r.K, BK);
  if (st != SQ_OK) return st;
  GradArgs p;
  p.M = static_cast<int32_t>(r.M);
  p.K = static_cast<int32_t>(r.K);
  p.num_n_tiles = static_cast<int32_t>((r.K + BN - 1) / BN);
  p.num_tiles = static_cast<int32_t>(plan.tiles);
  p.num_kb = static_cast<int32_t>((r.N + BK - 1) / BK);
  p.dx = r.dx;
  p.lddx = r.lddx;
  p.status = r.status;
  static bool attr_set[64] = {};
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64) return SQ_ERR_CUDA;
  if (!attr_set[dev]) {
    if (cudaFuncSetAttribute(input_grad_kernel<BN>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                             L::BYTES) != cudaSuccess)
      return SQ_ERR_CUDA;
    attr_set[dev] = true;
  }
  cudaLaunchConfig_t cfg = {};
  p.splits = plan.splits;
  cfg.gridDim = dim3(static_cast<unsigned>(2 * plan.splits * plan.clusters));
  cfg.blockDim = dim3(kGemmThreads);
  cfg.dynamicSmemBytes = L::BYTES;
  cfg.stream = stream;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = 2 * plan.splits;
  attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 2;
  if (cudaLaunchKernelEx(&cfg, input_grad_kernel<BN>, tmA, tmB, p) != cudaSuccess)
    return SQ_ERR_CUDA;
  return cudaGetLastError() == cudaSuccess ? SQ_OK : SQ_ERR_CUDA;
}

}  // namespace

size_t input_grad_workspace_bytes(int64_t N, int64_t K) {
  return static_cast<size_t>((N + 7) / 8 * 8) * static_cast<size_t>(K) * 2;
}

sq_status launch_input_grad(const InputGradRequest &r, cudaStream_t stream) {
  uint16_t *w = static_cast<uint16_t *>(r.workspace);
  constexpr int64_t kRows = kDeqLanes * kDeqRows;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>((r.K + 255) / 256),
                     static_cast<unsigned>((r.N + kRows - 1) / kRows));
  cfg.blockDim = dim3(kDeqThreads);
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  if (cudaLaunchKernelEx(&cfg, dequant_kernel, r.wq, r.s_w, r.d, r.N, r.K, r.seg, w, r.status) !=
      cudaSuccess)
    return SQ_ERR_CUDA;
  const InputGradPlan plan = input_grad_plan(r.M, r.N, r.K, sm_count());
  return plan.bn == 256 ? run_gemm<256>(r, w, plan, stream) : run_gemm<128>(r, w, plan, stream);
}

}  // namespace sq
