// Linear layer on 8-bit operands, on the 5th-generation tensor cores:
//   y[m][n] = x_scale[m] w_scale[n] sum_k x[m][k] w[n][k] + bias[n]
// x and w are e4m3, one scale for each row of x (token) and of w (output
// feature); products and sums are fp32 in TMEM, the scales and the bias are
// applied in fp32 and y is rounded once.
//
// linear_fp8_band_kernel: a CTA takes 128 rows of x (the MMA's rows; those
// past M are never stored) and a band of 64 output features, and streams both
// through a TMA ring of 128-byte K steps. Where the bands leave SMs idle K is
// split over a cluster whose CTAs add their fp32 tiles in rank order over
// distributed shared memory, so the result does not depend on which ran
// first. K past the end of a row reads as zeros.
//
// Measured, 12352 x 2048: one row and 64 rows 12.3 us a call (10.6 us as
// graph nodes, 2.4 TB/s): the ramp of 193 CTAs that each stream 128 KB.
//
// linear_fp8_tile_kernel: 256 x 256 tiles for prompts, each on a pair of CTAs
// (cta_group::2). An MMA of N = 256 holds the tensor pipe as long as its work
// takes (one of N = 64 more than twice as long), about 124 cycles a K step of
// 32. What it reads then counts: a CTA alone with 128 x 256 tiles writes and
// reads 24 KB of shared memory in that time, more than the 128 bytes a cycle
// there are (measured 81 us at 4096 x 12352 x 2048); the pair keeps half of w
// in either CTA, 16 KB. Persistent: warp 0 loads, warp 1 of the first CTA
// issues the MMAs, four warps of each scale and store the previous tile's 128
// rows out of the other half of TMEM, through swizzled shared memory and TMA,
// which also clips the edges (but for columns that end within 16 bytes). 4096 x
// 12352 x 2048 in bf16: 75.5 us, 2.74 PFLOP/s, the tensor pipe 80 % active.
#include <cuda.h>

#include <type_traits>

#include "gdn_common.cuh"
#include "gdn_internal.h"
#include "tc_common.cuh"
#include "tc_fp8.cuh"

namespace gdn {
namespace {

constexpr int kFM = 128;       // rows of x per tile
constexpr int kFBand = 64;     // output features per CTA
constexpr int kFK = 128;       // K per stage: one 128-byte swizzle atom
constexpr uint32_t kFWTile = kFBand * kFK;
constexpr int kFMaxStages = 12;
constexpr int kFThreads = 128;
constexpr int kFMaxSplits = 8;

struct BandPlan {
  int32_t splits, stages, box_rows;  // box_rows: rows of x per load
};

// the first n of eight elements, in 16-byte accesses where all of them are (dst on 16 bytes)
template <typename T>
__device__ __forceinline__ void store8(T* dst, const float* x, int n) {
  if (n >= 8) {
    alignas(16) T v[8];
#pragma unroll
    for (int e = 0; e < 8; ++e) v[e] = from_f32<T>(x[e]);
#pragma unroll
    for (int c = 0; c < (int)sizeof(T) / 2; ++c)
      reinterpret_cast<uint4*>(dst)[c] = reinterpret_cast<const uint4*>(v)[c];
  } else {
    for (int e = 0; e < 8 && e < n; ++e) dst[e] = from_f32<T>(x[e]);
  }
}

template <typename T>
__global__ void __launch_bounds__(kFThreads, 4)
    linear_fp8_band_kernel(const LinearFp8Args p, const BandPlan plan, const __grid_constant__ CUtensorMap tm_x,
                           const __grid_constant__ CUtensorMap tm_w) {
  extern __shared__ __align__(1024) unsigned char smem_raw[];
  unsigned char* sm = smem_raw + ((1024u - (smem_u32(smem_raw) & 1023u)) & 1023u);
  __shared__ __align__(8) uint64_t full[kFMaxStages], empty[kFMaxStages], done;
  __shared__ __align__(16) float s_scale[kFBand], s_bias[kFBand];
  __shared__ uint32_t s_tmem;
  __shared__ int s_abort;

  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int n0 = blockIdx.x * kFBand;
  const int64_t m0 = (int64_t)blockIdx.z * kFM;
  const int rows = p.M - m0 < kFM ? (int)(p.M - m0) : kFM;
  const int stages = plan.stages;
  const uint32_t x_bytes = (uint32_t)plan.box_rows * kFK;
  const uint32_t x_tile = (x_bytes + 1023) / 1024 * 1024, stage_bytes = x_tile + kFWTile;
  const int nk = (p.K + kFK - 1) / kFK;
  const int k_begin = (int)((int64_t)blockIdx.y * nk / plan.splits);
  const int k_len = (int)((int64_t)(blockIdx.y + 1) * nk / plan.splits) - k_begin;

  if (warp == 0) {
    tc::tmem_alloc(&s_tmem, kFBand);
    tc::tmem_relinquish();
  }
  if (tid == 0) {
    for (int s = 0; s < stages; ++s) {
      mbar_init(&full[s], 1);
      mbar_init(&empty[s], 1);
    }
    mbar_init(&done, 1);
    s_abort = 0;
    fence_mbar_init();
  }
  tc::fence_before_sync();
  __syncthreads();
  tc::fence_after_sync();
  const uint32_t tb = s_tmem;
  volatile int* abort_flag = &s_abort;
  uint32_t n_loads = 0;

  if (warp == 0 && lane == 0) {
    for (int i = 0; i < k_len; ++i) {
      const int s = i % stages;
      if (i >= stages && !mbar_wait_bounded(&empty[s], ((i / stages) - 1) & 1, abort_flag)) break;
      mbar_arrive_expect_tx(&full[s], x_bytes + kFWTile);
      ++n_loads;
      const int kx = (k_begin + i) * kFK;
      tc::tma_load_2d(sm + s * stage_bytes, &tm_x, kx, (int)m0, &full[s]);
      tc::tma_load_2d(sm + s * stage_bytes + x_tile, &tm_w, kx, n0, &full[s]);
    }
  } else if (warp == 1) {
    const uint32_t id = tc::idesc(tc::kE4M3, kFM, kFBand);
    const uint64_t d0 = tc::sdesc_sw128(smem_u32(sm));
    for (int i = 0; i < k_len; ++i) {
      const int s = i % stages;
      if (!__all_sync(0xffffffffu, mbar_wait_bounded(&full[s], (i / stages) & 1, abort_flag))) break;
      tc::fence_after_sync();
      const uint64_t dx = d0 + (uint64_t)((s * stage_bytes) >> 4);
      const uint64_t dw = d0 + (uint64_t)((s * stage_bytes + x_tile) >> 4);
#pragma unroll
      for (int ks = 0; ks < kFK / 32; ++ks)
        tc::mma_f8_elect(tb, tc::sdesc_at(dx, kFM, ks), tc::sdesc_at(dw, kFBand, ks), id, i > 0 || ks > 0);
      tc::mma_commit_elect(&empty[s]);
    }
    tc::mma_commit_elect(&done);
  } else if (warp >= 2) {
    // the band's scales and bias while the weights stream in
    static_assert(kFBand == 64, "one column for each thread of warps 2 and 3");
    const int c = tid - 64;
    const bool in = n0 + c < p.N;
    s_scale[c] = in ? __ldg(p.w_scale + n0 + c) : 0.f;
    s_bias[c] = in && p.bias != nullptr ? __ldg(p.bias + n0 + c) : 0.f;
  }

  // epilogue: thread (warp w, lane) holds row 32 w + lane of the accumulator
  const int m = 32 * warp + lane;
  const float my_scale = m < rows ? __ldg(p.x_scale + m0 + m) : 0.f;
  __syncwarp();
  const bool ok = mbar_wait_bounded(&done, 0, abort_flag) && !*abort_flag;
  __syncthreads();  // s_scale, s_bias
  tc::fence_after_sync();
  float v[kFBand];
  if (__all_sync(0xffffffffu, ok)) {
#pragma unroll
    for (int c = 0; c < kFBand / 16; ++c)
      tc::tmem_ld16(tb + ((uint32_t)(32 * warp) << 16) + 16 * c, *reinterpret_cast<float(*)[16]>(v + 16 * c));
    tc::tmem_wait_ld();
  } else {
#pragma unroll
    for (int e = 0; e < kFBand; ++e) v[e] = 0.f;
  }
  auto finish8 = [&](int r, int g8, float* x8, float xs) {
    const int n = n0 + 8 * g8, left = p.N - n;
    if (left <= 0) return;
#pragma unroll
    for (int e = 0; e < 8; ++e) x8[e] = fmaf(x8[e] * xs, s_scale[8 * g8 + e], s_bias[8 * g8 + e]);
    store8<T>(static_cast<T*>(p.y) + (m0 + r) * p.y_stride + n, x8, left);
  };
  if (plan.splits == 1) {
    if (m < rows && !*abort_flag)
#pragma unroll
      for (int g8 = 0; g8 < kFBand / 8; ++g8) finish8(m, g8, v + 8 * g8, my_scale);
  } else {
    // each split's fp32 tile in its own shared memory (the ring is idle:
    // every load it issued was consumed by an MMA that has completed),
    // 16-byte group c of row r at group c ^ (r % 16); every thread reaches
    // both cluster barriers, whatever happened before
    float* part = reinterpret_cast<float*>(sm);
    if (m < rows) {
#pragma unroll
      for (int c = 0; c < kFBand / 4; ++c)
        *reinterpret_cast<float4*>(part + m * kFBand + 4 * (c ^ (m & 15))) =
            make_float4(v[4 * c], v[4 * c + 1], v[4 * c + 2], v[4 * c + 3]);
    }
    cluster_arrive_release();
    cluster_wait_acquire();
    const int S = plan.splits, rank = (int)cluster_ctarank();
    const uint32_t base = smem_u32(part);
    if (!*abort_flag) {
      for (int u = rank * kFThreads + tid; u < rows * (kFBand / 8); u += S * kFThreads) {
        const int r = u >> 3, g8 = u & 7;
        const uint32_t o0 = (uint32_t)(r * kFBand + 4 * ((2 * g8) ^ (r & 15))) * 4u;
        const uint32_t o1 = (uint32_t)(r * kFBand + 4 * ((2 * g8 + 1) ^ (r & 15))) * 4u;
        const float xs = __ldg(p.x_scale + m0 + r);
        float x8[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
        for (int sp = 0; sp < S; ++sp) {
          const float4 a0 = ld_shared_cluster_f32x4(map_shared_rank(base + o0, (uint32_t)sp));
          const float4 a1 = ld_shared_cluster_f32x4(map_shared_rank(base + o1, (uint32_t)sp));
          x8[0] += a0.x, x8[1] += a0.y, x8[2] += a0.z, x8[3] += a0.w;
          x8[4] += a1.x, x8[5] += a1.y, x8[6] += a1.z, x8[7] += a1.w;
        }
        finish8(r, g8, x8, xs);
      }
    }
    cluster_arrive_release();
    cluster_wait_acquire();
  }

  // drain: every load this CTA issued has landed before TMEM is released
  tc::fence_before_sync();
  __syncthreads();
  if (warp == 0 && lane == 0) {
    for (uint32_t s = 0; s < (uint32_t)stages && s < n_loads; ++s) {
      const uint32_t uses = (n_loads - s + stages - 1) / stages;
      mbar_wait(&full[s], (uses - 1) & 1);
    }
  }
  __syncthreads();
  if (warp == 0) {
    tc::fence_after_sync();
    tc::tmem_dealloc(tb, kFBand);
  }
}

constexpr int kTN = 256;        // output features of a tile
constexpr int kTM = 256;        // rows of a tile, half in either CTA
constexpr int kTStages = 6;
constexpr uint32_t kTX = kFM * kFK, kTW = kTN / 2 * kFK, kTStage = kTX + kTW;  // of one CTA
constexpr int kTThreads = 192;  // loads, MMAs, four epilogue warps
constexpr uint32_t kTOut = 4096;  // one staged block: 32 rows of 128 bytes
constexpr uint32_t kTileSmem = kTStages * kTStage + 4 * kTOut;

template <typename T>
__global__ void __launch_bounds__(kTThreads, 1)
    linear_fp8_tile_kernel(const LinearFp8Args p, const __grid_constant__ CUtensorMap tm_x,
                           const __grid_constant__ CUtensorMap tm_w, const __grid_constant__ CUtensorMap tm_y) {
  extern __shared__ __align__(1024) unsigned char smem_raw[];
  unsigned char* sm = smem_raw + ((1024u - (smem_u32(smem_raw) & 1023u)) & 1023u);
  __shared__ __align__(8) uint64_t full[kTStages], empty[kTStages], acc_full[2], acc_empty[2];
  __shared__ __align__(16) float s_scale[2][kTN], s_bias[2][kTN];
  __shared__ uint32_t s_tmem;
  __shared__ int s_abort;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int nk = (p.K + kFK - 1) / kFK;
  const int m_tiles = (int)((p.M + kTM - 1) / kTM), n_tiles = (p.N + kTN - 1) / kTN;
  const int tiles = m_tiles * n_tiles;
  const int rank = (int)cluster_ctarank(), pair = blockIdx.x / 2, pairs = gridDim.x / 2;

  if (warp == 0) tc::tmem_alloc_pair(&s_tmem, 2 * kTN);
  if (tid == 0) {
    for (int s = 0; s < kTStages; ++s) {
      mbar_init(&full[s], 1);
      mbar_init(&empty[s], 1);
    }
    for (int a = 0; a < 2; ++a) {
      mbar_init(&acc_full[a], 1);
      mbar_init(&acc_empty[a], 8);  // the epilogue warps of both CTAs
    }
    s_abort = 0;
    fence_mbar_init();
  }
  tc::fence_before_sync();
  __syncthreads();
  // both CTAs' barriers and TMEM are there before either is used by the other
  cluster_arrive_release();
  cluster_wait_acquire();
  tc::fence_after_sync();
  const uint32_t tb = s_tmem;
  volatile int* abort_flag = &s_abort;
  uint32_t loads = 0;

  // the row tiles of a column tile run side by side: its rows of w are read
  // once from memory, x stays in L2
  if (warp == 0) {
    if (lane == 0) {
      for (int tile = pair; tile < tiles; tile += pairs) {
        const int m0 = (tile % m_tiles) * kTM + rank * kFM, n0 = (tile / m_tiles) * kTN + rank * (kTN / 2);
        for (int k = 0; k < nk; ++k, ++loads) {
          const int s = loads % kTStages;
          if (loads >= kTStages && !mbar_wait_bounded(&empty[s], (loads / kTStages - 1) & 1, abort_flag)) goto loaded;
          // both CTAs' loads complete on the first one's barrier
          const uint32_t bar = map_shared_rank(smem_u32(&full[s]), 0);
          if (rank == 0) mbar_arrive_expect_tx(&full[s], 2 * kTStage);
          tc::tma_load_2d_pair(sm + s * kTStage, &tm_x, k * kFK, m0, bar);
          tc::tma_load_2d_pair(sm + s * kTStage + kTX, &tm_w, k * kFK, n0, bar);
        }
      }
    }
  loaded:
    __syncwarp();
  } else if (warp == 1 && rank == 0) {
    const uint32_t id = tc::idesc(tc::kE4M3, kTM, kTN);
    const uint64_t d0 = tc::sdesc_sw128(smem_u32(sm));
    uint32_t i = 0;
    int n = 0;
    bool ok = true;
    for (int tile = pair; ok && tile < tiles; tile += pairs, ++n) {
      const int a = n & 1;
      if (n >= 2) ok = __all_sync(0xffffffffu, mbar_wait_bounded(&acc_empty[a], (n / 2 - 1) & 1, abort_flag));
      if (!ok) break;
      for (int k = 0; k < nk; ++k, ++i) {
        const int s = i % kTStages;
        ok = __all_sync(0xffffffffu, mbar_wait_bounded(&full[s], (i / kTStages) & 1, abort_flag));
        if (!ok) break;
        tc::fence_after_sync();
        const uint64_t dx = d0 + (uint64_t)((s * kTStage) >> 4), dw = dx + (uint64_t)(kTX >> 4);
#pragma unroll
        for (int ks = 0; ks < kFK / 32; ++ks)
          tc::mma_f8_pair_elect(tb + a * kTN, tc::sdesc_at(dx, kFM, ks), tc::sdesc_at(dw, kTN / 2, ks), id, k > 0 || ks > 0);
        tc::mma_commit_pair_elect(&empty[s]);
      }
      tc::mma_commit_pair_elect(&acc_full[a]);
    }
  } else if (warp >= 2) {
    const int qd = warp & 3;  // TMEM lane quadrant
    constexpr int kCols = 128 / (int)sizeof(T);  // columns of a staged block
    unsigned char* at = sm + kTStages * kTStage + (warp - 2) * kTOut;
    int n = 0;
    for (int tile = pair; tile < tiles; tile += pairs, ++n) {
      const int a = n & 1;
      const int64_t m0 = (int64_t)(tile % m_tiles) * kTM + rank * kFM;
      const int n0 = (tile / m_tiles) * kTN;
      // this tile's scales and bias; the buffers are two tiles apart in use
      for (int c = tid - 64; c < kTN; c += 128) {
        const bool in = n0 + c < p.N;
        s_scale[a][c] = in ? __ldg(p.w_scale + n0 + c) : 0.f;
        s_bias[a][c] = in && p.bias != nullptr ? __ldg(p.bias + n0 + c) : 0.f;
      }
      const int64_t m = m0 + 32 * qd + lane;
      const float xs = m < p.M ? __ldg(p.x_scale + m) : 0.f;
      asm volatile("bar.sync 1, 128;" ::: "memory");
      // after a wait that gave up the warps still meet at the barrier above
      if (!__all_sync(0xffffffffu, mbar_wait_bounded(&acc_full[a], (n / 2) & 1, abort_flag))) continue;
      tc::fence_after_sync();
      const uint32_t tq = tb + ((uint32_t)(32 * qd) << 16) + a * kTN;
      for (int c0 = 0; c0 < kTN; c0 += kCols) {
        float v[kCols];
#pragma unroll
        for (int c = 0; c < kCols; c += 16) tc::tmem_ld16(tq + c0 + c, *reinterpret_cast<float(*)[16]>(v + c));
        tc::tmem_wait_ld();
        if (c0 + kCols == kTN) {  // the accumulator is read
          tc::fence_before_sync();
          __syncwarp();
          if (lane == 0) mbar_arrive_cluster(map_shared_rank(smem_u32(&acc_empty[a]), 0));
        }
        if (n0 + c0 >= p.N || m0 + 32 * qd >= p.M) continue;
#pragma unroll
        for (int c = 0; c < kCols; c += 4) {
          const float4 ws = *reinterpret_cast<const float4*>(&s_scale[a][c0 + c]);
          const float4 b = *reinterpret_cast<const float4*>(&s_bias[a][c0 + c]);
          v[c] = fmaf(v[c] * xs, ws.x, b.x);
          v[c + 1] = fmaf(v[c + 1] * xs, ws.y, b.y);
          v[c + 2] = fmaf(v[c + 2] * xs, ws.z, b.z);
          v[c + 3] = fmaf(v[c + 3] * xs, ws.w, b.w);
        }
        // TMA clips a row at 16 bytes, not at an element: a last block that
        // ends within them is stored from the registers
        const int left = p.N - (n0 + c0);
        if (left < kCols && left % (16 / (int)sizeof(T)) != 0) {
          if (m < p.M) {
            T* row = static_cast<T*>(p.y) + m * p.y_stride + n0 + c0;
#pragma unroll
            for (int c = 0; c < kCols; c += 8) store8<T>(row + c, v + c, left - c);
          }
          continue;
        }
        if (lane == 0) bulk_wait_read_all();  // the last block's store has read the buffer
        __syncwarp();
#pragma unroll
        for (int c = 0; c < 8; ++c) {
          alignas(16) T x[16 / sizeof(T)];
#pragma unroll
          for (int i = 0; i < 16 / (int)sizeof(T); ++i) x[i] = from_f32<T>(v[c * (16 / sizeof(T)) + i]);
          *reinterpret_cast<uint4*>(at + lane * 128 + ((c ^ (lane & 7)) << 4)) = *reinterpret_cast<const uint4*>(x);
        }
        fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) {
          tc::tma_store_2d(&tm_y, n0 + c0, (int)m0 + 32 * qd, at);
          bulk_commit();
        }
      }
    }
    if (lane == 0) bulk_wait_all();
  }

  // no load or MMA may be in flight, and nothing of the other CTA under way to
  // this one, when the CTA ends: the last loads into each stage, then the pair
  tc::fence_before_sync();
  __syncthreads();
  if (tid == 0) {
    for (uint32_t s = 0; s < (uint32_t)kTStages && s < loads; ++s) {
      const uint32_t last = ((loads - s + kTStages - 1) / kTStages - 1) & 1;
      if (rank == 0) mbar_wait(&full[s], last);
      mbar_wait_bounded(&empty[s], last, abort_flag);
    }
  }
  __syncthreads();
  cluster_arrive_release();
  cluster_wait_acquire();
  if (warp == 0) {
    tc::fence_after_sync();
    tc::tmem_dealloc_pair(tb, 2 * kTN);
  }
}

int sm_count() {
  int dev = 0, n = 0;
  if (cudaGetDevice(&dev) != cudaSuccess ||
      cudaDeviceGetAttribute(&n, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess || n <= 0)
    return 148;
  return n;
}

template <typename T>
cudaError_t launch_band(const LinearFp8Args& p, const void* x, int64_t x_stride, const void* w, cudaStream_t stream) {
  BandPlan plan;
  plan.box_rows = p.M < kFM ? (int32_t)p.M : kFM;
  const CUtensorMapDataType u8 = CU_TENSOR_MAP_DATA_TYPE_UINT8;
  CUtensorMap mx, mw;
  if (!tc::make_map_2d(&mx, x, p.M, p.K, x_stride, 1, u8, kFK, (uint32_t)plan.box_rows, CU_TENSOR_MAP_SWIZZLE_128B) ||
      !tc::make_map_2d(&mw, w, p.N, p.K, p.K, 1, u8, kFK, kFBand, CU_TENSOR_MAP_SWIZZLE_128B,
                       CU_TENSOR_MAP_L2_PROMOTION_L2_256B))
    return cudaErrorInvalidValue;
  const int bands = (p.N + kFBand - 1) / kFBand, nk = (p.K + kFK - 1) / kFK;
  const int64_t tiles = (p.M + kFM - 1) / kFM;
  // Two CTAs of 96 KB an SM (12352 x 2048, 64 rows: 10.6 us; three CTAs of 64 KB
  // 11.5, four of 48 KB 17.9) and as many K splits as still run in one wave,
  // each of two K steps at least, of eight from 32 rows on, whose fp32 tiles are
  // as large as a K step (2048 x 4096, 128 rows: eight splits 13.2 us, four 9.7;
  // one row 7.5 and 8.2). A cluster lies in one GPC of 18 or 20 SMs, so
  // fewer of them run at once than the SMs have places (3808 x 3984, three
  // rows: 60 clusters of four 9.3 us, of five 15.0).
  // Where the bands fill several waves, four CTAs of 54 KB in all, so that one
  // starts and stores under the others' streams (65536 x 2048: one row 27.7 us
  // against 41.9, 128 rows 37.0 against 42.4; three CTAs 33.5 and 36.8).
  const bool waves = bands * tiles >= 4 * sm_count();
  const auto clusters = [](int s) { return s == 1 ? INT64_MAX : s == 2 ? 152 : 8ll * (36 / s); };
  int splits = nk / (p.M < 32 ? 2 : 8);
  if (splits > kFMaxSplits) splits = kFMaxSplits;
  while (splits > 1 && bands * tiles > clusters(splits)) --splits;
  plan.splits = splits < 1 ? 1 : splits;
  const uint32_t x_tile = ((uint32_t)plan.box_rows * kFK + 1023) / 1024 * 1024, stage_bytes = x_tile + kFWTile;
  const uint32_t extra = (kFM * kFK - x_tile) + 1024;  // the MMA reads kFM rows from a stage's start; alignment
  const int fit = (int)((waves ? 54 * 1024 - extra : 96 * 1024) / stage_bytes);
  plan.stages = fit < 2 ? 2 : (fit < kFMaxStages ? fit : kFMaxStages);  // two hold a split's fp32 tile, too
  const uint32_t smem = (uint32_t)plan.stages * stage_bytes + extra;
  auto kern = linear_fp8_band_kernel<T>;
  cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
  if (e != cudaSuccess) return e;
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3((unsigned)bands, (unsigned)plan.splits, (unsigned)tiles);
  cfg.blockDim = dim3(kFThreads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = 1;
  attr[0].val.clusterDim.y = (unsigned)plan.splits;
  attr[0].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = plan.splits > 1 ? 1 : 0;
  e = cudaLaunchKernelEx(&cfg, kern, p, plan, mx, mw);
  return e != cudaSuccess ? e : cudaGetLastError();
}

template <typename T>
cudaError_t launch_tile(const LinearFp8Args& p, const void* x, int64_t x_stride, const void* w, cudaStream_t stream) {
  const CUtensorMapDataType u8 = CU_TENSOR_MAP_DATA_TYPE_UINT8;
  const CUtensorMapDataType yt = sizeof(T) == 4                            ? CU_TENSOR_MAP_DATA_TYPE_FLOAT32
                                 : std::is_same<T, __nv_bfloat16>::value ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16
                                                                         : CU_TENSOR_MAP_DATA_TYPE_FLOAT16;
  CUtensorMap mx, mw, my;
  if (!tc::make_map_2d(&mx, x, p.M, p.K, x_stride, 1, u8, kFK, kFM, CU_TENSOR_MAP_SWIZZLE_128B,
                       CU_TENSOR_MAP_L2_PROMOTION_L2_256B) ||
      !tc::make_map_2d(&mw, w, p.N, p.K, p.K, 1, u8, kFK, kTN / 2, CU_TENSOR_MAP_SWIZZLE_128B,
                       CU_TENSOR_MAP_L2_PROMOTION_L2_256B) ||
      !tc::make_map_2d(&my, p.y, p.M, p.N, p.y_stride, sizeof(T), yt, 128 / sizeof(T), 32, CU_TENSOR_MAP_SWIZZLE_128B))
    return cudaErrorInvalidValue;
  auto kern = linear_fp8_tile_kernel<T>;
  constexpr int smem = (int)kTileSmem + 1024;
  const cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
  if (e != cudaSuccess) return e;
  const int64_t tiles = (p.M + kTM - 1) / kTM * ((p.N + kTN - 1) / kTN);
  const int pairs = sm_count() / 2;
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3(2 * (unsigned)(tiles < pairs ? tiles : pairs));
  cfg.blockDim = dim3(kTThreads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = 2;
  attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  const cudaError_t r = cudaLaunchKernelEx(&cfg, kern, p, mx, mw, my);
  return r != cudaSuccess ? r : cudaGetLastError();
}

template <typename T>
cudaError_t launch_t(const LinearFp8Args& p, const void* x, int64_t x_stride, const void* w, cudaStream_t stream) {
  // tiles from where they keep half the SMs busy; below, and for one row tile
  // (a stream of w), bands and K splits give more CTAs
  const int64_t tiles = (p.M + kTM - 1) / kTM * ((p.N + kTN - 1) / kTN);
  if (p.M > kFM && 4 * tiles >= sm_count() && tiles <= INT32_MAX / 2) return launch_tile<T>(p, x, x_stride, w, stream);
  return launch_band<T>(p, x, x_stride, w, stream);
}

}  // namespace

cudaError_t launch_linear_fp8(const LinearFp8Args& p, const void* x, int64_t x_stride, const void* w,
                              int32_t out_dtype, cudaStream_t stream) {
  switch (out_dtype) {
    case GDN_F16: return launch_t<__half>(p, x, x_stride, w, stream);
    case GDN_BF16: return launch_t<__nv_bfloat16>(p, x, x_stride, w, stream);
    case GDN_F32: return launch_t<float>(p, x, x_stride, w, stream);
    default: return cudaErrorInvalidValue;
  }
}

}  // namespace gdn

GDN_DEFINE_ERROR_READER(linear_fp8)
