// Softmax attention on the 5th-generation tensor cores (f16, bf16).
//
// An item is two tiles of 128 rows (token, query head of the group), A and B,
// that share the keys' tiles of 128. For both, tile after tile:
//   S = Q K^T        both from shared memory, fp32 into TMEM
//   P = exp2(S scale log2 e - M)     a thread per row, 16 bits, into TMEM
//   O += P V         P from TMEM, V read transposed, fp32 in TMEM
// A row lies in a lane of TMEM, so its maximum and sum are one thread's and
// need no exchange. M follows the row's maximum only where that has grown by
// more than 8 (in log2) since: then the row's O and sum are rescaled, which is
// rare; else the weights are up to 2^8, as exact as below 1. The sum is of the
// weights before their rounding to 16 bits.
//
// TMEM's 512 columns hold O of both tiles (256), P of both (128) and one S.
// The tiles take turns in it: a row's thread reads all of its scores into
// registers at once, so S is free again long before the softmax is done, and
// the scores of the other tile, then the tile's own next ones, are made under
// it. With two S, each with its P in its place, the next scores of a tile had
// to wait for its O += P V: a chain of softmax and both products. Now both
// tiles take 2550 cycles at head_dim 128, of which the products are 2048.
//
// Warps 0 to 3 are A's rows, 4 to 7 B's; two issue the products, one hands out
// the pieces of work (attn_common.cuh) and loads (Q once an item, K and V
// through a ring of tiles each), one looks through masked tiles of V: a
// masked weight is 0, but 0 times what is not finite would reach rows that do
// not see it. So rows of V that nobody sees become 0, and in rows that only
// some see what is not finite is replaced by 0 and added, at the end, to the
// rows that do see it.
//
// One warp issues the scores, another O += P V: the tensor cores take a few
// products ahead from each, and an issuing warp is held until they do, so that
// with one warp for both whatever the other kind waited for was looked at late.
// A tile's next scores go first, then its O: its rows wait for the scores, and
// for O only when their next weights are done.
//
// Rounding. The weights go to 16 bits because the tensor cores multiply them by
// V in the type of V; the error that adds is that of the output's own rounding
// again (0.0021 of the outputs' norm in bf16, where the exact result rounded
// has 0.0016). The tensor cores cut their fp32 sums off, up to 1.5 2^-24 of O
// for each step of 16 keys, always towards zero: 2^-11 once a CTA takes 131,072
// keys in a row, 0.006 at 2^20 (measured; f16, no workspace).
//
// Measured (as graph nodes): one prompt of 4096 tokens, 32 query heads and 8
// key heads of 128, 105 us, 1.31 PFLOP/s of the visible pairs, the tensor pipe
// 62 % active; 32,768 tokens, 16 and 2 heads, 1.95 PFLOP/s. 64 single tokens on
// caches of up to 8192 keys 174 us, 6.3 TB/s. What bounds it: on prompts of
// head_dim 128 the tensor cores, and the end of an item and the start of the
// next (5,900 cycles from its last weights to the next scores); on caches of
// head_dim 128 memory. At head_dim 64 and below nothing is full (tensor pipe 40
// %, exponentials 40 %, issue 45 %): a tile is a chain from scores to weights
// of about 1,750 cycles whatever head_dim is, and the two warps of rows that a
// scheduler has do not hide it (2,070 cycles for both tiles, products 1,024).
// Items of at most 128 rows (single tokens) have half A alone.
//
// A wait that gives up raises the CTA's abort flag; every role then leaves its
// loop at once.
#include <cuda.h>
#include <stddef.h>

#include "attn_common.cuh"
#include "tc_common.cuh"

namespace gdn {
namespace {

constexpr int kBR = 128;          // rows of a tile
constexpr int kBK = 128;          // keys of a tile
constexpr int kBThreads = 384;
constexpr int kBScores = 8, kBLoad = 9, kBOut = 10, kBCheck = 11;  // warps
constexpr int kBRing = 4;         // pieces handed out ahead
constexpr int kBTakers = 11;      // warps that take each piece: all but the one that loads
constexpr float kBGrow = 8.f;     // log2 by which a weight may exceed 1
constexpr float kBFar = 65536.f;  // scaled scores from which on the maximum is taken off before they are scaled

template <int D>
struct TcGeom {
  static constexpr int kBoxes = (D + 63) / 64;
  static constexpr uint32_t kTile = kBoxes * kBK * 128;  // bytes
  static constexpr int kStages = kBoxes == 2 ? 2 : 4;  // of each ring
  static constexpr uint32_t kK = 2 * kTile, kV = kK + kStages * kTile;
  static constexpr uint32_t kOut = kV + kStages * kTile;  // 4 KB for each warp of rows
  static constexpr uint32_t kSmem = kOut + 8 * 4096;
};

// TMEM columns: S, P of both tiles (64 each), O of both (128 each)
constexpr uint32_t kColS = 0, kColP = 128, kColO = 256, kCols = 512;

struct BShared {
  // the rings of K, which the scores' warp empties, and of V, which the
  // outputs' warp and the one that looks through it do: whoever waits for a
  // tile also has to give it back, so no phase of a barrier goes by unseen
  uint64_t k_full[4], k_empty[4], v_full[4], v_empty[4], v_ok[4];
  // p_ready: the four warps' weights, and the scores of the tile after
  uint64_t q_full[2], q_empty[2], s_full[2], s_free, p_ready[2], o_done[2];
  uint64_t piece_full[kBRing], piece_empty[kBRing];
  AttnPiece piece[kBRing];
  AttnPlan plan;
  int abort, loads;  // (side by side: wait_for_piece); tiles that were asked for
  uint32_t tmem;
};
static_assert(offsetof(BShared, loads) == offsetof(BShared, abort) + 4, "wait_for_piece");

// the tile [k][mn] of 16-bit elements with k as the contraction (MN-major,
// 128-byte swizzle), boxes of 64 mn columns kTile / kBoxes apart; 16 of k
// advance it by 2048 bytes
__device__ __forceinline__ uint64_t sdesc_v(uint32_t smem_addr) {
  uint64_t d = 0;
  d |= (uint64_t)((smem_addr & 0x3FFFF) >> 4);
  d |= (uint64_t)((kBK * 128) >> 4) << 16;
  d |= (uint64_t)(1024 >> 4) << 32;
  d |= (uint64_t)1 << 46;
  d |= (uint64_t)2 << 61;
  return d;
}
constexpr uint32_t kTransB = 1u << 16;

__device__ __forceinline__ void tmem_ld32(uint32_t taddr, float* v) {
  uint32_t r[32];
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x32.b32 "
      "{%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,"
      "%16,%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31}, [%32];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]),
        "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15]), "=r"(r[16]),
        "=r"(r[17]), "=r"(r[18]), "=r"(r[19]), "=r"(r[20]), "=r"(r[21]), "=r"(r[22]), "=r"(r[23]), "=r"(r[24]),
        "=r"(r[25]), "=r"(r[26]), "=r"(r[27]), "=r"(r[28]), "=r"(r[29]), "=r"(r[30]), "=r"(r[31])
      : "r"(taddr));
#pragma unroll
  for (int i = 0; i < 32; ++i) v[i] = __uint_as_float(r[i]);
}

__device__ __forceinline__ void prefetch_map(const void* map) {
  asm volatile("prefetch.tensormap [%0];" ::"l"(map) : "memory");
}
__device__ __forceinline__ void tma_load_3d(void* dst, const void* map, int x, int y, int z, uint64_t* bar) {
  asm volatile(
      "cp.async.bulk.tensor.3d.shared::cluster.global.tile.mbarrier::complete_tx::bytes "
      "[%0], [%1, {%2, %3, %4}], [%5];" ::"r"(smem_u32(dst)),
      "l"(map), "r"(x), "r"(y), "r"(z), "r"(smem_u32(bar))
      : "memory");
}
__device__ __forceinline__ void tma_load_4d(void* dst, const void* map, int x, int y, int z, int w, uint64_t* bar) {
  asm volatile(
      "cp.async.bulk.tensor.4d.shared::cluster.global.tile.mbarrier::complete_tx::bytes "
      "[%0], [%1, {%2, %3, %4, %5}], [%6];" ::"r"(smem_u32(dst)),
      "l"(map), "r"(x), "r"(y), "r"(z), "r"(w), "r"(smem_u32(bar))
      : "memory");
}

// Consecutive k-steps issued by one elected lane of a converged warp, their
// descriptors counted up here: one election and one pair of descriptors for
// all of them. Four steps of both operands K-major (32 bytes each)...
template <int STEPS>
__device__ __forceinline__ void mma_ss(uint32_t d_tmem, uint64_t a, uint64_t b, uint32_t id, bool accumulate) {
  static_assert(STEPS == 2 || STEPS == 4, "within a 128-byte atom");
  if constexpr (STEPS == 4)
    asm volatile(
        "{\n\t.reg .pred e, p;\n\t.reg .b64 a1, a2, a3, b1, b2, b3;\n\t"
        "elect.sync _|e, 0xffffffff;\n\tsetp.ne.b32 p, %4, 0;\n\t"
        "add.s64 a1, %1, 2;\n\tadd.s64 a2, %1, 4;\n\tadd.s64 a3, %1, 6;\n\t"
        "add.s64 b1, %2, 2;\n\tadd.s64 b2, %2, 4;\n\tadd.s64 b3, %2, 6;\n\t"
        "@e tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n\t"
        "@e tcgen05.mma.cta_group::1.kind::f16 [%0], a1, b1, %3, 1;\n\t"
        "@e tcgen05.mma.cta_group::1.kind::f16 [%0], a2, b2, %3, 1;\n\t"
        "@e tcgen05.mma.cta_group::1.kind::f16 [%0], a3, b3, %3, 1;\n\t}" ::"r"(d_tmem),
        "l"(a), "l"(b), "r"(id), "r"((uint32_t)accumulate)
        : "memory");
  else
    asm volatile(
        "{\n\t.reg .pred e, p;\n\t.reg .b64 a1, b1;\n\t"
        "elect.sync _|e, 0xffffffff;\n\tsetp.ne.b32 p, %4, 0;\n\t"
        "add.s64 a1, %1, 2;\n\tadd.s64 b1, %2, 2;\n\t"
        "@e tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n\t"
        "@e tcgen05.mma.cta_group::1.kind::f16 [%0], a1, b1, %3, 1;\n\t}" ::"r"(d_tmem),
        "l"(a), "l"(b), "r"(id), "r"((uint32_t)accumulate)
        : "memory");
}
// ... and four of A from TMEM (8 columns each), B MN-major (2048 bytes).
__device__ __forceinline__ void mma_ts4(uint32_t d_tmem, uint32_t a_tmem, uint64_t b, uint32_t id, bool accumulate) {
  asm volatile(
      "{\n\t.reg .pred e, p;\n\t.reg .b64 b1, b2, b3;\n\t.reg .b32 a1, a2, a3;\n\t"
      "elect.sync _|e, 0xffffffff;\n\tsetp.ne.b32 p, %4, 0;\n\t"
      "add.u32 a1, %1, 8;\n\tadd.u32 a2, %1, 16;\n\tadd.u32 a3, %1, 24;\n\t"
      "add.s64 b1, %2, 128;\n\tadd.s64 b2, %2, 256;\n\tadd.s64 b3, %2, 384;\n\t"
      "@e tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t"
      "@e tcgen05.mma.cta_group::1.kind::f16 [%0], [a1], b1, %3, 1;\n\t"
      "@e tcgen05.mma.cta_group::1.kind::f16 [%0], [a2], b2, %3, 1;\n\t"
      "@e tcgen05.mma.cta_group::1.kind::f16 [%0], [a3], b3, %3, 1;\n\t}" ::"r"(d_tmem),
      "r"(a_tmem), "l"(b), "r"(id), "r"((uint32_t)accumulate)
      : "memory");
}

__device__ __forceinline__ float exp2_fast(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

// A bounded wait that sleeps in the barrier; false when *abort_flag is set or
// after kWaitLimitNs, and then it sets the flag. (In a few instructions: there
// are many of these, and what a CTA runs must fit the instruction cache.)
__device__ __forceinline__ bool wait_for(uint64_t* bar, uint32_t parity, int* abort_flag) {
  uint32_t ok;
  asm volatile(
      "{\n\t.reg .pred p, q;\n\t.reg .b64 t0, t1;\n\t.reg .b32 f;\n\t"
      "mbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2, %3;\n\t"
      "@p bra DONE;\n\t"
      "mov.u64 t0, %%globaltimer;\n"
      "AGAIN:\n\t"
      "mbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2, %3;\n\t"
      "@p bra DONE;\n\t"
      "ld.volatile.shared.b32 f, [%4];\n\t"
      "setp.ne.b32 q, f, 0;\n\t"
      "@q bra DONE;\n\t"
      "mov.u64 t1, %%globaltimer;\n\t"
      "sub.u64 t1, t1, t0;\n\t"
      "setp.lt.u64 q, t1, %5;\n\t"
      "@q bra AGAIN;\n\t"
      "mov.b32 f, 1;\n\t"
      "st.volatile.shared.b32 [%4], f;\n"
      "DONE:\n\t"
      "selp.u32 %0, 1, 0, p;\n\t}"
      : "=r"(ok)
      : "r"(smem_u32(bar)), "r"(parity), "r"(20000u), "r"(smem_u32(abort_flag)), "l"(kWaitLimitNs)
      : "memory");
  return ok != 0;
}

// The same for a piece of work, which the loading warp hands out behind the
// last tile of the one before: a half without rows waits for it as long as the
// other half's tiles take, and a long cache's take more than any fixed time. So
// the limit counts from the last tile that was asked for (an int behind
// *abort_flag); there are finitely many, and the loading warp's own waits have
// the plain limit, so this one ends too.
__device__ __forceinline__ bool wait_for_piece(uint64_t* bar, uint32_t parity, int* abort_flag) {
  uint32_t ok;
  asm volatile(
      "{\n\t.reg .pred p, q;\n\t.reg .b64 t0, t1;\n\t.reg .b32 f, n0, n1;\n\t"
      "mbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2, %3;\n\t"
      "@p bra DONE;\n\t"
      "mov.u64 t0, %%globaltimer;\n\t"
      "ld.volatile.shared.b32 n0, [%4+4];\n"
      "AGAIN:\n\t"
      "mbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2, %3;\n\t"
      "@p bra DONE;\n\t"
      "ld.volatile.shared.b32 f, [%4];\n\t"
      "setp.ne.b32 q, f, 0;\n\t"
      "@q bra DONE;\n\t"
      "mov.u64 t1, %%globaltimer;\n\t"
      "ld.volatile.shared.b32 n1, [%4+4];\n\t"
      "setp.ne.b32 q, n1, n0;\n\t"
      "@q mov.u64 t0, t1;\n\t"
      "mov.b32 n0, n1;\n\t"
      "sub.u64 t1, t1, t0;\n\t"
      "setp.lt.u64 q, t1, %5;\n\t"
      "@q bra AGAIN;\n\t"
      "mov.b32 f, 1;\n\t"
      "st.volatile.shared.b32 [%4], f;\n"
      "DONE:\n\t"
      "selp.u32 %0, 1, 0, p;\n\t}"
      : "=r"(ok)
      : "r"(smem_u32(bar)), "r"(parity), "r"(20000u), "r"(smem_u32(abort_flag)), "l"(kWaitLimitNs)
      : "memory");
  return ok != 0;
}

template <typename T>
struct Half;
template <>
struct Half<__nv_bfloat16> {
  static constexpr uint32_t kFormat = tc::kBF16;
  // log2 that the weights are scaled by
  static constexpr float kLift = 0.f;
  __device__ __forceinline__ static uint32_t pack(float lo, float hi) {
    uint32_t r;
    asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
    return r;
  }
  // 0 x + c: NaN where x is not finite, c elsewhere (c a zero of either sign, or NaN)
  __device__ __forceinline__ static uint32_t zero_times(uint32_t x, uint32_t c) {
    uint32_t r;
    asm("fma.rn.bf16x2 %0, %1, %2, %3;" : "=r"(r) : "r"(x), "r"(0u), "r"(c));
    return r;
  }
};
template <>
struct Half<__half> {
  static constexpr uint32_t kFormat = tc::kF16;
  // fp16's smallest normal weight would be 2^-14: 2^7 of its range above 2^8
  // is moved below
  static constexpr float kLift = 7.f;
  __device__ __forceinline__ static uint32_t pack(float lo, float hi) {
    uint32_t r;
    asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
    return r;
  }
  __device__ __forceinline__ static uint32_t zero_times(uint32_t x, uint32_t c) {
    uint32_t r;
    asm("fma.rn.f16x2 %0, %1, %2, %3;" : "=r"(r) : "r"(x), "r"(0u), "r"(c));
    return r;
  }
};

// Tiles of keys that half h (A or B) of the piece has, from t0 on.
__device__ __forceinline__ int half_tiles(const AttnArgs& p, const AttnPiece& w, int h) {
  const int tokens = p.item / 2, first = h * tokens;
  if (first >= w.tokens) return 0;
  const int last = (first + tokens < w.tokens ? first + tokens : w.tokens) - 1;
  const int seen = attn_sees(w, last);
  int end = seen / kBK + (seen % kBK != 0);
  end = end < w.t1 ? end : w.t1;
  return end > w.t0 ? end - w.t0 : 0;
}
// Whether some row of the item does not see all of the tile.
__device__ __forceinline__ bool masked_tile(int least, int t) { return (int64_t)(t + 1) * kBK > least; }

template <typename T, int D>
__global__ void __launch_bounds__(kBThreads, 1)
    attn_tc_kernel(const AttnArgs p, const __grid_constant__ CUtensorMap tm_q, const __grid_constant__ CUtensorMap tm_k,
                   const __grid_constant__ CUtensorMap tm_v) {
  using G = TcGeom<D>;
  extern __shared__ __align__(1024) unsigned char smem_raw[];
  unsigned char* sm = smem_raw + ((1024u - (smem_u32(smem_raw) & 1023u)) & 1023u);
  __shared__ BShared sh;
  const int tid = threadIdx.x, lane = tid & 31, warp = __shfl_sync(0xffffffffu, tid >> 5, 0);

  if (warp == kBScores) {
    tc::tmem_alloc(&sh.tmem, kCols);
    tc::tmem_relinquish();
  }
  if (tid == 32) {
    prefetch_map(&tm_q);
    prefetch_map(&tm_k);
    prefetch_map(&tm_v);
  }
  if (tid == 0) {
    for (int i = 0; i < G::kStages; ++i) {
      mbar_init(&sh.k_full[i], 1);
      mbar_init(&sh.k_empty[i], 1);
      mbar_init(&sh.v_full[i], 1);
      mbar_init(&sh.v_empty[i], 2);
      mbar_init(&sh.v_ok[i], 1);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(&sh.q_full[i], 1);
      mbar_init(&sh.q_empty[i], 1);
      mbar_init(&sh.s_full[i], 1);
      mbar_init(&sh.p_ready[i], 5);
      mbar_init(&sh.o_done[i], 1);
    }
    mbar_init(&sh.s_free, 4);
    for (int i = 0; i < kBRing; ++i) {
      mbar_init(&sh.piece_full[i], 1);
      mbar_init(&sh.piece_empty[i], kBTakers);
    }
    sh.abort = sh.loads = 0;
    fence_mbar_init();
  }
  if (tid < 2 && p.part_o != nullptr) p.part_at[2 * blockIdx.x + tid] = make_int4(kAttnWhole, 0, 0, 0);
  attn_plan<kBK, kBThreads>(p, reinterpret_cast<int64_t*>(sm), &sh.plan);  // (nothing is loaded yet)
  fence_proxy_async_smem();
  tc::fence_before_sync();
  __syncthreads();
  tc::fence_after_sync();
  const uint32_t tb = __shfl_sync(0xffffffffu, sh.tmem, 0);
  const auto wait = [&](uint64_t* bar, uint32_t parity) { return wait_for(bar, parity, &sh.abort); };
  // piece i of the CTA, for a whole warp; false: there is none
  const auto take = [&](int i, AttnPiece* w) {
    const bool ok = wait_for_piece(&sh.piece_full[i % kBRing], (i / kBRing) & 1, &sh.abort);
    *w = sh.piece[i % kBRing];
    return __all_sync(0xffffffffu, ok) && w->tokens != 0;
  };
  const auto give = [&](int i) {
    __syncwarp();
    if (lane == 0) mbar_arrive(&sh.piece_empty[i % kBRing]);
  };

  // The softmax holds a row of scores in registers. Of the 168 a thread that
  // the block has, 384 x 168 = 64512, two groups of 128 threads take 208 and
  // one keeps 80: 63488.
  if (warp >= 8) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 80;");
    if (warp == kBLoad) {
      // ----------------------------------------------------- pieces and loads
      uint32_t n_k = 0, n_v = 0, n_q[2] = {0, 0};
      const uint32_t q_bytes = (uint32_t)(G::kBoxes * 128 * (p.item / 2) * p.group);
      bool ok = true;
      const auto load = [&](const CUtensorMap* map, unsigned char* ring, uint64_t* full, uint64_t* empty, uint32_t& n,
                            int kh, int row) {
        const uint32_t st = n % G::kStages, round = n / G::kStages;
        ok = ok && (round == 0 || wait(&empty[st], (round - 1) & 1));
        if (!ok) return;
        ++n;
        *(volatile int*)&sh.loads = (int)(n_k + n_v);
        mbar_arrive_expect_tx(&full[st], G::kTile);
        for (int b = 0; b < G::kBoxes; ++b)
          tma_load_3d(ring + st * G::kTile + b * kBK * 128, map, 64 * b, kh, row, &full[st]);
      };
      const auto load_k = [&](int kh, int row) { load(&tm_k, sm + G::kK, sh.k_full, sh.k_empty, n_k, kh, row); };
      const auto load_v = [&](int kh, int row) { load(&tm_v, sm + G::kV, sh.v_full, sh.v_empty, n_v, kh, row); };
      AttnWalk<kBK> walk;
      walk.start(p, sh.plan, lane);
      for (int i = 0;; ++i) {
        const AttnPiece w = walk.next(p);
        if (i >= kBRing && !__all_sync(0xffffffffu, wait(&sh.piece_empty[i % kBRing], (i / kBRing - 1) & 1))) break;
        if (lane == 0) {
          sh.piece[i % kBRing] = w;
          mbar_arrive(&sh.piece_full[i % kBRing]);
        }
        if (w.tokens == 0) break;
        if (lane == 0 && ok) {
          const auto load_q = [&](int h) {
            if (half_tiles(p, w, h) == 0) return;
            ok = ok && (n_q[h] == 0 || wait(&sh.q_empty[h], (n_q[h] - 1) & 1));
            if (!ok) return;
            ++n_q[h];
            mbar_arrive_expect_tx(&sh.q_full[h], q_bytes);
            for (int b = 0; b < G::kBoxes; ++b)
              tma_load_4d(sm + h * G::kTile + b * kBR * 128, &tm_q, 64 * b, 0, w.kh, w.q0 + h * (p.item / 2),
                          &sh.q_full[h]);
          };
          for (int t = w.t0; ok && t < w.t1; ++t) {
            if (t == w.t0) load_q(0);
            load_k(w.kh, w.k0 + t * kBK);
            if (t == w.t0) load_q(1);
            else load_v(w.kh, w.k0 + (t - 1) * kBK);
          }
          if (ok && w.t0 < w.t1) load_v(w.kh, w.k0 + (w.t1 - 1) * kBK);
        }
        __syncwarp();
      }
      if (lane == 0) {
        // nothing may be in flight when the CTA ends: neither a copy nor the
        // arrival that gives a tile back
        const auto over = [&](uint64_t* full, uint64_t* empty, uint32_t n) {
          for (uint32_t u = n > G::kStages ? n - G::kStages : 0; u < n; ++u) {
            mbar_wait(&full[u % G::kStages], (u / G::kStages) & 1);
            wait(&empty[u % G::kStages], (u / G::kStages) & 1);
          }
        };
        over(sh.k_full, sh.k_empty, n_k);
        over(sh.v_full, sh.v_empty, n_v);
        for (int h = 0; h < 2; ++h)
          if (n_q[h] > 0) {
            mbar_wait(&sh.q_full[h], (n_q[h] - 1) & 1);
            wait(&sh.q_empty[h], (n_q[h] - 1) & 1);
          }
      }
    } else if (warp == kBScores || warp == kBOut) {
      // ------------------------------------------------------------ products
      // (a whole warp goes through this, and one lane issues: addresses stay
      // in uniform registers, where one lane's branch took twice as long. For
      // the same end what is read from shared memory is taken from one lane,
      // so that the compiler knows it to be the same in all.)
      const auto all = [&](bool x) { return __all_sync(0xffffffffu, x); };
      const auto same = [&](int x) { return __shfl_sync(0xffffffffu, x, 0); };
      uint32_t n_kv = 0, n[2] = {0, 0};
      bool ok = true;
      // the stage of the ring's next tile, once it is there
      const auto next_tile = [&](uint64_t* full) {
        const uint32_t st = n_kv % G::kStages;
        ok = all(wait(&full[st], (n_kv / G::kStages) & 1)) && ok;
        ++n_kv;
        return st;
      };
      if (warp == kBScores) {
        const uint32_t id = tc::idesc(Half<T>::kFormat, kBR, kBK);
        const uint64_t dq = tc::sdesc_sw128(smem_u32(sm)), dk = tc::sdesc_sw128(smem_u32(sm + G::kK));
        uint32_t n_s = 0;
        for (int i = 0; ok; ++i) {
          AttnPiece w;
          if (!take(i, &w)) break;
          const int tiles = same(w.t1 - w.t0), na = same(half_tiles(p, w, 0)), nb = same(half_tiles(p, w, 1));
          for (int j = 0; ok && j < tiles; ++j) {
            const uint32_t st = next_tile(sh.k_full);
#pragma unroll
            for (int h = 0; h < 2; ++h) {
              if (j >= (h ? nb : na)) continue;
              if (j == 0) {
                ok = ok && all(wait(&sh.q_full[h], n[h] & 1));
                ++n[h];
              }
              ok = ok && (n_s == 0 || all(wait(&sh.s_free, (n_s - 1) & 1)));
              ++n_s;
              if (!ok) continue;
              tc::fence_after_sync();
              const uint64_t a = dq + (h * G::kTile >> 4), b = dk + (st * G::kTile >> 4);
              constexpr uint32_t next = kBK * 128 >> 4;  // the second 64 columns
              mma_ss<D == 32 ? 2 : 4>(tb + kColS, a, b, id, false);
              if (D > 64) mma_ss<D == 96 ? 2 : 4>(tb + kColS, a + next, b + next, id, true);
              tc::mma_commit_elect(&sh.s_full[h]);
              if (j > 0 && lane == 0) mbar_arrive(&sh.p_ready[h]);  // O of the tile before may come now
              if (j + 1 == (h ? nb : na)) tc::mma_commit_elect(&sh.q_empty[h]);
            }
            if (ok) tc::mma_commit_elect(&sh.k_empty[st]);
          }
          give(i);
        }
      } else {
        const uint32_t id = tc::idesc(Half<T>::kFormat, kBR, D) | kTransB;
        const uint64_t dv = sdesc_v(smem_u32(sm + G::kV));
        uint32_t ok_bits = 0;
        for (int i = 0; ok; ++i) {
          AttnPiece w;
          if (!take(i, &w)) break;
          const int tiles = same(w.t1 - w.t0), na = same(half_tiles(p, w, 0)), nb = same(half_tiles(p, w, 1));
          const int least = same(attn_sees(w, 0)), t0 = same(w.t0);
          for (int j = 0; ok && j < tiles; ++j) {
            const uint32_t st = next_tile(sh.v_full);
            if (ok && masked_tile(least, t0 + j)) {
              ok = all(wait(&sh.v_ok[st], (ok_bits >> st) & 1));
              ok_bits ^= 1u << st;
            }
#pragma unroll
            for (int h = 0; h < 2; ++h) {
              if (j >= (h ? nb : na)) continue;
              ok = ok && all(wait(&sh.p_ready[h], n[h] & 1));
              ++n[h];
              if (!ok) continue;
              tc::fence_after_sync();
              const uint64_t b = dv + (st * G::kTile >> 4);
              mma_ts4(tb + kColO + 128 * h, tb + kColP + 64 * h, b, id, j > 0);
              mma_ts4(tb + kColO + 128 * h, tb + kColP + 64 * h + 32, b + (8192 >> 4), id, true);
              tc::mma_commit_elect(&sh.o_done[h]);
            }
            if (ok) tc::mma_commit_elect(&sh.v_empty[st]);
          }
          give(i);
        }
      }
    } else if (warp == kBCheck) {
      // ------------------------------------------------- masked tiles of v
      uint32_t n_v = 0;
      for (int i = 0;; ++i) {
        AttnPiece w;
        if (!take(i, &w)) break;
        const int least = attn_sees(w, 0), most = attn_sees(w, w.tokens - 1);
        for (int t = w.t0; t < w.t1; ++t) {
          const uint32_t st = n_v % G::kStages;
          if (!__all_sync(0xffffffffu, wait(&sh.v_full[st], (n_v / G::kStages) & 1))) break;
          ++n_v;
          if (!masked_tile(least, t)) {
            if (lane == 0) mbar_arrive(&sh.v_empty[st]);
            continue;
          }
          unsigned char* v = sm + G::kV + st * G::kTile;
          const int base = t * kBK, from = least > base ? least - base : 0;  // rows from which some row sees no more
          bool hit = false;
          constexpr int kC = 8 * G::kBoxes, kR = 32 / kC;  // 16-byte chunks of a row, rows an access
          const int c16 = lane % kC, some = lane / kC;
          unsigned char* col = v + (c16 >> 3) * kBK * 128;
          const auto place = [&](int row) {
            return reinterpret_cast<uint4*>(col + row * 128 + (((c16 & 7) ^ (row & 7)) << 4));
          };
          const int until = most - base < kBK ? most - base : kBK;
          // Eight accesses in flight. 0 times anything finite adds nothing; nearly
          // always there is nothing to store.
#pragma unroll 1
          for (int r0 = from + some; r0 < until; r0 += 8 * kR) {
            uint4 x[8];
            uint32_t any = 0;
#pragma unroll
            for (int k = 0; k < 8; ++k) x[k] = r0 + kR * k < until ? *place(r0 + kR * k) : make_uint4(0, 0, 0, 0);
#pragma unroll
            for (int k = 0; k < 8; ++k)
#pragma unroll
              for (int j = 0; j < 4; ++j) any = Half<T>::zero_times((&x[k].x)[j], any);
            if ((any & 0x7fff7fffu) == 0) continue;
            hit = true;
#pragma unroll 1
            for (int r = r0; r < until && r < r0 + 8 * kR; r += kR) {
              uint4 y = *place(r);
#pragma unroll
              for (int j = 0; j < 4; ++j) {
                uint32_t& e = (&y.x)[j];
                const uint32_t m = Half<T>::zero_times(e, 0);
                if (m & 0x7fffu) e &= 0xffff0000u;
                if (m & 0x7fff0000u) e &= 0x0000ffffu;
              }
              *place(r) = y;
            }
          }
#pragma unroll 4
          for (int r = until + some; r < kBK; r += kR) *place(r) = make_uint4(0, 0, 0, 0);
          if (hit) sh.piece[i % kBRing].bad = 1;
          fence_proxy_async_smem();
          __syncwarp();
          if (lane == 0) {
            mbar_arrive(&sh.v_ok[st]);
            mbar_arrive(&sh.v_empty[st]);
          }
        }
        give(i);
      }
    }
  } else {
    asm volatile("setmaxnreg.inc.sync.aligned.u32 208;");
    // ------------------------------------------------------------- softmax
    const int h = warp >> 2, qd = warp & 3, row = 32 * qd + lane;
    const uint32_t ts = tb + ((uint32_t)(32 * qd) << 16) + kColS, tp = ts + kColP + 64 * h;
    const uint32_t to = tb + ((uint32_t)(32 * qd) << 16) + kColO + 128 * h;
    const float sc = p.scale * kAttnLog2e, grows = fminf(kBGrow / sc, 3.4e38f);
    const int half = p.item / 2, row_token = h * half + row / p.group, member = row % p.group;
    const bool row_used = row < half * p.group;
    uint32_t n_s = 0;  // tiles so far
    bool alive = true;
    // this warp's weights are there; where the tile has no scores to come, so are those
    const auto ready = [&](bool last) {
      if (lane != 0) return;
      mbar_arrive(&sh.p_ready[h]);
      if (last && qd == 0) mbar_arrive(&sh.p_ready[h]);
    };
    // whether O has taken the weights of tile n of this half (from 1 on)
    const auto o_done = [&](uint32_t n) {
      if (n > 0) alive = __all_sync(0xffffffffu, wait(&sh.o_done[h], (n - 1) & 1));
      tc::fence_after_sync();
      return alive;
    };
    for (int i = 0;; ++i) {
      AttnPiece w;
      if (!take(i, &w)) break;
      const int at = row_token;  // of the item
      const bool valid = row_used && at < w.tokens;
      const int sees = valid ? attn_sees(w, at) : 0;
      const int n = half_tiles(p, w, h);
      const bool some = __any_sync(0xffffffffu, valid);
      const int least = (int)__reduce_min_sync(0xffffffffu, valid ? (unsigned)sees : 0x7fffffffu);
      // M: the largest score so far (or a little less), not scaled. base: what
      // makes a scaled score its weight's exponent, kLift less the scaled M.
      // Rounded, it is off by 2^-24 of itself, for all of a row's weights alike,
      // which the division by their sum undoes; but 2^30 would move them by 2^5,
      // out of what 16 bits hold. So from kBFar on M is taken off the scores
      // before they are scaled, which is exact next to it, and kLift is added.
      float M = -INFINITY, base = 0.f, plus = 0.f;
      bool far = false;  // such a row is among the warp's
      const auto base_of = [&](float m) { return m == -INFINITY ? 0.f : fmaf(-m, sc, Half<T>::kLift); };
      float2 sum = make_float2(0.f, 0.f);
      for (int j = 0; j < n; ++j) {
        alive = __all_sync(0xffffffffu, wait(&sh.s_full[h], n_s & 1));
        if (!alive) break;
        ++n_s;
        tc::fence_after_sync();
        if (!some) {  // no row of this warp counts
          __syncwarp();
          if (lane == 0) mbar_arrive(&sh.s_free);
          // (the other warps' weights of the tile before are counted)
          if (!o_done(n_s - 1)) break;
          ready(j + 1 == n);
          continue;
        }
        float s[kBK];
#pragma unroll
        for (int c = 0; c < kBK; c += 32) tmem_ld32(ts + c, s + c);
        tc::tmem_wait_ld();
        tc::fence_before_sync();
        __syncwarp();
        if (lane == 0) mbar_arrive(&sh.s_free);
        const int t = w.t0 + j;
        if (masked_tile(least, t)) {
          const int lim = sees - t * kBK;
#pragma unroll
          for (int c = 0; c < kBK; ++c)
            if (c >= lim) s[c] = -INFINITY;
        }
        float top[4] = {s[0], s[1], s[2], s[3]};
#pragma unroll
        for (int c = 4; c < kBK; c += 8)
#pragma unroll
          for (int e = 0; e < 4; ++e) top[e] = fmaxf(fmaxf(top[e], s[c + e]), c + 4 + e < kBK ? s[c + 4 + e] : top[e]);
        const float high = fmaxf(fmaxf(top[0], top[1]), fmaxf(top[2], top[3]));
        // rare: a maximum that has grown (in a first tile, from nothing), or rows far off
        const bool grow = high - M > grows;
        if (__any_sync(0xffffffffu, grow) || far) {
          float f = 1.f;
          if (grow) {
            const float next = base_of(high);
            f = exp2_fast(fabsf(next) >= kBFar || M == -INFINITY ? (M - high) * sc : next - base);
            M = high;
            base = next;
          }
          if (j > 0 && __any_sync(0xffffffffu, grow)) {
            if (!o_done(n_s - 1)) break;
            sum = make_float2(sum.x * f, sum.y * f);
#pragma unroll 1
            for (int c = 0; c < D; c += 16) {
              float o[16];
              tc::tmem_ld16(to + c, o);
              tc::tmem_wait_ld();
#pragma unroll
              for (int e = 0; e < 16; ++e) o[e] *= f;
              tc::tmem_st16(to + c, o);
            }
          }
          plus = base;
          far = __any_sync(0xffffffffu, fabsf(base) >= kBFar);
          if (far) {
            float off = 0.f;
            if (fabsf(base) >= kBFar) off = M, plus = Half<T>::kLift;
#pragma unroll
            for (int c = 0; c < kBK; ++c) s[c] -= off;
          }
        }
        const float2 sc2 = make_float2(sc, sc), base2 = make_float2(plus, plus), one = make_float2(1.f, 1.f);
        uint32_t r[kBK / 2];
#pragma unroll
        for (int c = 0; c < kBK / 2; ++c) {
          float2 x = fma2(make_float2(s[2 * c], s[2 * c + 1]), sc2, base2);
          x.x = exp2_fast(x.x);
          x.y = exp2_fast(x.y);
          sum = fma2(x, one, sum);
          r[c] = Half<T>::pack(x.x, x.y);
        }
        // O has taken the weights of the tile before, whose place these take
        if (!o_done(n_s - 1)) break;
#pragma unroll
        for (int c = 0; c < kBK / 2; c += 16) tc::tmem_st16u(tp + c, *reinterpret_cast<uint32_t(*)[16]>(r + c));
        tc::tmem_wait_st();
        tc::fence_before_sync();
        __syncwarp();
        ready(j + 1 == n);
      }
      if (!alive) break;
      // ---- the outputs
      if (some) {
        if (n > 0 && !o_done(n_s)) break;
        const float l = sum.x + sum.y, top = M == -INFINITY ? M : -base;
        if (n > 0 && *(volatile int*)&sh.piece[i % kBRing].bad != 0) {
          // what the look through V took out of rows that this one sees
          const int item_least = attn_sees(w, 0);
          const int first = max(item_least, w.t0 * kBK), last = (int)min((int64_t)sees, (int64_t)w.t1 * kBK);
#pragma unroll 1
          for (int c = 0; c < D; c += 16) {
            float o[16];
            tc::tmem_ld16(to + c, o);
            tc::tmem_wait_ld();
            const T* v = static_cast<const T*>(p.v) + (int64_t)w.kh * D + c;
#pragma unroll 1
            for (int k = first; valid && k < last; ++k)
#pragma unroll
              for (int e = 0; e < 16; ++e) {
                const float x = to_f32(v[(int64_t)(w.k0 + k) * p.v_stride + e]);
                if (!isfinite(x)) o[e] += x;
              }
            __syncwarp();
            tc::tmem_st16(to + c, o);
          }
          tc::tmem_wait_st();
        }
        int64_t to_row = 0;
        AttnScale f{1.f, 0.f};
        float* part_out = attn_part_out(p, w.causal);
        if (valid) {
          const int64_t token = w.q0 + at;
          const int head = attn_head(p, w.kh, member);
          if (w.part != kAttnWhole) {
            const int64_t slot = attn_slot(blockIdx.x, w.part);
            const int64_t slot_row = slot * p.part_rows + at * p.group + member;
            p.part_ml[slot_row] = make_float2(top, l);
            to_row = slot_row * D;
          } else {
            float* lse = attn_lse(p, w.causal);
            f = attn_scale(top, l, lse != nullptr);
            to_row = (token * p.Hq + head) * D;
            if (lse != nullptr) lse[token * p.Hq + head] = f.lse;
          }
        }
        // 64 or 128 bytes of each row at a time through shared memory, so that
        // they are stored side by side (from the lanes' rows a store of 16 bytes
        // each touches 32 lines)
        const bool wide = w.part != kAttnWhole || part_out != nullptr;  // fp32
        unsigned char* stage = sm + G::kOut + warp * 4096;
        const unsigned live = __ballot_sync(0xffffffffu, valid);
        const auto store = [&](auto* y, auto as) {
          using E = decltype(as);
          constexpr int kCols = 32, kBytes = kCols * (int)sizeof(E);
          constexpr int kLanes = kBytes / 16, kRows = 32 / kLanes;  // lanes a row, rows an access
          int64_t at_row[32 / kRows];
#pragma unroll
          for (int k = 0; k < 32 / kRows; ++k) at_row[k] = __shfl_sync(0xffffffffu, to_row, kRows * k + lane / kLanes);
          // 16-byte chunk e of row r: eight lanes of a row or of eight rows use all banks
          const auto chunk = [&](int r, int e) {
            const int x = kLanes == 8 ? r & 7 : r >> 1 & 3;
            return reinterpret_cast<uint4*>(stage + r * kBytes + ((e ^ x) << 4));
          };
#pragma unroll 1
          for (int c = 0; c < D; c += kCols) {
            float o[kCols];
            if (n > 0) {
              tmem_ld32(to + c, o);
              tc::tmem_wait_ld();
            } else {
#pragma unroll
              for (int e = 0; e < kCols; ++e) o[e] = 0.f;
            }
#pragma unroll
            for (int e = 0; e < kCols; e += 2) {
              const float2 y = fma2(make_float2(o[e], o[e + 1]), make_float2(f.factor, f.factor), make_float2(-0.f, -0.f));
              o[e] = y.x, o[e + 1] = y.y;
            }
            __syncwarp();
#pragma unroll
            for (int e = 0; e < kLanes; ++e) {
              const float* y4 = o + 4 * e;
              const float* y8 = o + 8 * e;
              if constexpr (sizeof(E) == 4)
                *chunk(lane, e) = make_uint4(__float_as_uint(y4[0]), __float_as_uint(y4[1]), __float_as_uint(y4[2]),
                                             __float_as_uint(y4[3]));
              else
                *chunk(lane, e) = make_uint4(Half<T>::pack(y8[0], y8[1]), Half<T>::pack(y8[2], y8[3]),
                                             Half<T>::pack(y8[4], y8[5]), Half<T>::pack(y8[6], y8[7]));
            }
            __syncwarp();
#pragma unroll
            for (int k = 0; k < 32 / kRows; ++k) {
              const int r = kRows * k + lane / kLanes, e = lane % kLanes;
              const uint4 x = *chunk(r, e);
              if (live >> r & 1) *reinterpret_cast<uint4*>(y + at_row[k] + c + e * (16 / (int)sizeof(E))) = x;
            }
          }
        };
        if (wide) store(w.part != kAttnWhole ? p.part_o : part_out, 0.f);
        else store(static_cast<T*>(p.out), T());
        if (tid == 0 && w.part != kAttnWhole)
          p.part_at[attn_slot(blockIdx.x, w.part)] = make_int4(w.part + 4 * w.causal, w.q0, w.tokens, w.kh);
      }
      give(i);
    }
  }
  tc::fence_before_sync();
  __syncthreads();
  if (tid == 0 && sh.abort) record_device_error(GDN_ERR_TIMEOUT);
  if (warp == kBScores) {
    tc::fence_after_sync();
    tc::tmem_dealloc(tb, kCols);
  }
}

bool make_map(CUtensorMap* m, const void* base, CUtensorMapDataType dt, int rank, const cuuint64_t* dims,
              const cuuint64_t* strides, const cuuint32_t* box) {
  const tc::EncodeTiledFn fn = tc::encode_fn();
  const cuuint32_t one[4] = {1, 1, 1, 1};
  return fn != nullptr && fn(m, dt, (cuuint32_t)rank, const_cast<void*>(base), dims, strides, box, one,
                             CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
                             CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

template <typename T, int D>
cudaError_t run(const AttnArgs& p, CUtensorMapDataType dt, int grid, cudaStream_t stream) {
  CUtensorMap mq, mk, mv;
  const cuuint64_t g = (cuuint64_t)p.group, Hk = (cuuint64_t)p.Hk, head = D * 2;
  // q as [token][key head][member of its group][D], whichever of the two lie
  // side by side
  const bool tiled = p.map == GDN_MAP_TILED;
  const cuuint64_t qd[4] = {D, g, Hk, (cuuint64_t)p.T};
  const cuuint64_t qs[3] = {tiled ? Hk * head : head, tiled ? head : g * head, (cuuint64_t)p.q_stride * 2};
  const cuuint32_t qb[4] = {64, (cuuint32_t)g, 1, (cuuint32_t)(p.item / 2)};
  const cuuint64_t kd[3] = {D, Hk, (cuuint64_t)(p.kv_rows > 0 ? p.kv_rows : 1)};
  const cuuint64_t ks[2] = {head, (cuuint64_t)p.k_stride * 2}, vs[2] = {head, (cuuint64_t)p.v_stride * 2};
  const cuuint32_t kb[3] = {64, 1, kBK};
  // (a cache of no rows is never read)
  if (!make_map(&mq, p.q, dt, 4, qd, qs, qb) || !make_map(&mk, p.kv_rows > 0 ? p.k : p.q, dt, 3, kd, ks, kb) ||
      !make_map(&mv, p.kv_rows > 0 ? p.v : p.q, dt, 3, kd, vs, kb))
    return cudaErrorInvalidValue;
  constexpr int smem = (int)TcGeom<D>::kSmem + 1024;
  const cudaError_t e = cudaFuncSetAttribute(attn_tc_kernel<T, D>, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
  if (e != cudaSuccess) return e;
  attn_tc_kernel<T, D><<<grid, kBThreads, smem, stream>>>(p, mq, mk, mv);
  return cudaGetLastError();
}
template <typename T>
cudaError_t run_dim(const AttnArgs& p, CUtensorMapDataType dt, int32_t D, int grid, cudaStream_t stream) {
  switch (D) {
    case 32: return run<T, 32>(p, dt, grid, stream);
    case 64: return run<T, 64>(p, dt, grid, stream);
    case 96: return run<T, 96>(p, dt, grid, stream);
    default: return run<T, 128>(p, dt, grid, stream);
  }
}

}  // namespace

int attn_tc_rows() { return kBR; }

cudaError_t launch_attn_tc(const AttnArgs& p, int32_t dtype, int32_t D, int grid, cudaStream_t stream) {
  if (dtype == GDN_F16) return run_dim<__half>(p, CU_TENSOR_MAP_DATA_TYPE_FLOAT16, D, grid, stream);
  return run_dim<__nv_bfloat16>(p, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, D, grid, stream);
}

}  // namespace gdn

GDN_DEFINE_ERROR_READER(attn_tc)
