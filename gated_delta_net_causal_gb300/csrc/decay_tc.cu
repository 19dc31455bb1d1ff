// Linear attention with a decay for each head over packed sequences, on the
// 5th-generation tensor cores (bf16 activations, head_dim 128): 64 tokens at
// a time, with the state S[j][i] fp32 in registers.
//
// With G_t the sum of the chunk's log decays up to token t and G_n up to its
// last one, the recurrence over a chunk is
//   P[t][s]  = scale e^(G_t - G_s) q_t . k_s   for s <= t, else 0
//   o_t[j]   = scale e^(G_t) sum_i S[j][i] q_t[i]  +  sum_s P[t][s] v_s[j]
//   S[j][i] <- e^(G_n) S[j][i] + sum_s v_s[j] (e^(G_n - G_s) k_s[i])
// so no chunk waits on anything but the state before it. The products, with
// value rows j or tokens t on the 128 or 64 MMA rows:
//   scores  [t][s] = Q K^T               both tiles as TMA loads them
//   O1      [j][t] = S Q^T               S from TMEM as bf16 hi + lo
//   O2      [j][t] = V^T P^T             V read transposed, P as bf16 hi + lo
//   dS      [j][i] = V^T K'              K' = e^(G_n - G_s) k as bf16 hi + mid + lo
// q, k and v are exact in bf16. What is added to the state has three bf16
// parts (2^-24 of a factor), as the state is kept in fp32. S and P only reach
// the outputs: two parts (2^-17 of a factor). One part would be off by 2^-8 of
// the terms' magnitudes, which is far more than the rounding of a 16-bit out
// where terms cancel; the second costs 6 % with the gated norm and 14 %
// without (88 and 553 us with one), most of it the conversions of S. The MMAs
// cut their sums off at fp32's last bits, so the smallest parts are added
// first: with them last sums of positive terms came out up to 2^-18.6 of
// themselves too small, so up to 2^-22.
//
// A pipeline of one CTA per SM, whose warps hand each other tiles through
// mbarriers instead of meeting at barriers. Sixteen warps compute; per chunk c
// they go through
//   P(c)   from the scores, which were issued a chunk ahead
//   K'(c)  in its parts
//   the outputs, from O1(c) and O2(c)
//   S      from dS(c), and its bf16 copy for O1(c + 1)
// while the tensor cores run O2(c), dS(c), the scores of c + 1 and O1(c + 1),
// each as soon as its operands are there: O2 runs under K', dS under the
// outputs, the rest under everything. One warp issues the MMAs, one loads, one
// sums the log decays and one stores the outputs and loads z into their
// places. q, k, v, z and the outputs have two stages, and TMEM holds every
// accumulator side by side. The outputs leave TMEM as 8 x 8 blocks, are normed
// and gated in registers, transposed in shared memory and stored by TMA.
//
// What bounds it: a chunk of a head takes about 4800 cycles (8 x 1024 tokens,
// 64 heads, no gate; 6100 with the gated norm, whose exponentials and
// reciprocals are 1000 of the MUFU's), a chain of phases of the same warps in
// which no unit is full. 8 ragged prompts of 34,482 tokens in all, 64 heads:
// 631 us, 2360 GB/s; one of 4096 tokens, 32 heads: 93 us. With one part of S
// and P, the same chunks with two CTAs an SM that meet at barriers took 630
// and 105 us against 564 and 88.
//
// Exponents are differences of sums of up to 64 log decays, which a decay of
// -100 a token makes large where the difference is small; the sums are held
// as two floats each.
//
// A NaN or an infinity in v times a masked P (0) would reach tokens before
// it: such elements of v are replaced by 0 before the product and make NaN in
// their value row of the outputs from their token on, and of the state.
//
// Segments (decay_common.cuh) run as in decay_scan.cu: a first pass
// (kPLocal) adds up dS alone, with two stages of K' and of the accumulator
// too; the second starts each segment from what those before it leave.
//
// A wait that gives up raises the CTA's abort flag; every role then runs
// through its remaining waits at once and the kernel ends.
#include <cuda.h>

#include "decay_common.cuh"
#include "tc_common.cuh"

namespace gdn {
namespace {

constexpr int kTc = 64;  // tokens per chunk
constexpr int kTd = 128;

// Descriptor of a tile [k][mn] of 16-bit elements read with k as the
// contraction (MN-major, 128-byte swizzle): boxes of 64 mn columns 8 KB apart,
// eight k rows in 1024 bytes, so that 16 of k advance it by 2048.
__device__ __forceinline__ uint64_t sdesc_mn128(uint32_t smem_addr) {
  uint64_t d = 0;
  d |= (uint64_t)((smem_addr & 0x3FFFF) >> 4);
  d |= (uint64_t)(8192 >> 4) << 16;
  d |= (uint64_t)(1024 >> 4) << 32;
  d |= (uint64_t)1 << 46;
  d |= (uint64_t)2 << 61;
  return d;
}
constexpr uint32_t kTransA = 1u << 15, kTransB = 1u << 16;

// Four 8 x 8 blocks of 16-bit elements between shared memory and registers,
// transposed: lane l gives the address of row l % 8 of block l / 8, and its
// register m holds elements (2 (l % 4), l / 4) and (2 (l % 4) + 1, l / 4) of
// block m as (shared row, shared column).
__device__ __forceinline__ void ldmatrix_t4(uint32_t addr, uint32_t (&r)[4]) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0, %1, %2, %3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr)
               : "memory");
}
__device__ __forceinline__ void stmatrix_t4(uint32_t addr, const uint32_t (&r)[4]) {
  asm volatile("stmatrix.sync.aligned.m8n8.x4.trans.shared.b16 [%0], {%1, %2, %3, %4};" ::"r"(addr), "r"(r[0]),
               "r"(r[1]), "r"(r[2]), "r"(r[3])
               : "memory");
}

__device__ __forceinline__ float exp2_fast(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
// two floats to packed bf16 (x in the low half)
__device__ __forceinline__ uint32_t pack2(float2 a) {
  uint32_t r;
  asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(a.y), "f"(a.x));
  return r;
}
__device__ __forceinline__ float2 unpack2(uint32_t r) {
  return make_float2(__uint_as_float(r << 16), __uint_as_float(r & 0xffff0000u));
}
// the same, leaving in a what the rounding dropped
__device__ __forceinline__ uint32_t split2(float2& a) {
  const uint32_t r = pack2(a);
  a = fma2(unpack2(r), make_float2(-1.f, -1.f), a);
  return r;
}
// the same with the hi part cut off instead of rounded: no conversion, and
// what is left is exact too
__device__ __forceinline__ uint32_t cut2(float2& a) {
  const uint32_t x = __float_as_uint(a.x), y = __float_as_uint(a.y);
  a = fma2(make_float2(__uint_as_float(x & 0xffff0000u), __uint_as_float(y & 0xffff0000u)), make_float2(-1.f, -1.f), a);
  return __byte_perm(x, y, 0x7632);
}
__device__ __forceinline__ float2 mul2(float2 a, float b) { return fma2(a, make_float2(b, b), make_float2(-0.f, -0.f)); }

// a + b as two floats
struct Two {
  float hi, lo;
};
__device__ __forceinline__ Two add2(Two a, Two b) {
  const float s = a.hi + b.hi;
  const float t = s - a.hi;
  const float e = (a.hi - (s - t)) + (b.hi - t);
  const float l = e + (a.lo + b.lo);
  const float h = s + l;
  return Two{h, l - (h - s)};
}
constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.69314718055994531f;
constexpr float kLog2eLo = 1.9259629911e-8f;  // log2(e) less its fp32 rounding
__device__ __forceinline__ Two to_log2(float g) {
  const float h = g * kLog2e;
  return Two{h, fmaf(g, kLog2e, -h) + g * kLog2eLo};
}

constexpr int kPCompute = 16;  // compute warps: TMEM lane quadrant warp % 4, column quarter warp / 4
constexpr int kPMma = 16, kPLoad = 17, kPGates = 18, kPStore = 19;
constexpr int kPThreads = 32 * 20;
enum { kPWhole = 0, kPLocal = 1 };

// shared memory, from a 1024-byte boundary; tiles of 64 tokens x 128 columns
// are two boxes of 64 columns, 128-byte swizzled rows
constexpr uint32_t kPTile = 16384;
constexpr uint32_t kPQ = 0;            // [2]
constexpr uint32_t kPK = 2 * kPTile;   // [2] K, then K' hi in place
constexpr uint32_t kPV = 4 * kPTile;   // [2]
constexpr uint32_t kPMid = 6 * kPTile;  // K' mid, K' lo
constexpr uint32_t kPP = 8 * kPTile;   // P and its low part; first pass: the second K' mid and lo
constexpr uint32_t kPO = 9 * kPTile;   // [2] z, then the outputs in its place
constexpr uint32_t kPSmem = 11 * kPTile;
__device__ __forceinline__ uint32_t mid_at(int stage) { return stage ? kPO : kPMid; }

// TMEM columns
constexpr uint32_t kPColS = 0;     // S hi (64 packed columns), S lo (64)
constexpr uint32_t kPColSc = 128;  // scores
constexpr uint32_t kPColO2 = 192;
constexpr uint32_t kPColO1 = 256;
constexpr uint32_t kPColKv = 320;  // dS; first pass: at 0 and 128
constexpr uint32_t kPCols = 512;

// 16 lanes x 16 columns: thread lane holds rows lane/4 and lane/4 + 8, columns
// 8 c + 2 (lane % 4) and the next, at v[4 c], v[4 c + 1] and v[4 c + 2], v[4 c + 3]
__device__ __forceinline__ void tmem_ld_16x16(uint32_t taddr, float (&v)[8]) {
  uint32_t r[8];
  asm volatile("tcgen05.ld.sync.aligned.16x256b.x2.b32 {%0,%1,%2,%3,%4,%5,%6,%7}, [%8];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7])
               : "r"(taddr));
#pragma unroll
  for (int i = 0; i < 8; ++i) v[i] = __uint_as_float(r[i]);
}

struct TcShared {
  Two G[4][kTc];     // by chunk % 4: sums of log2 decays
  float E[4][kTc];   // scale e^(G_t)
  float dk[4][kTc];  // e^(G_n - G_s), 0 past the chunk's tokens
  Decay whole[4];    // e^(G_n)
  int bad[4][kTd];   // first token with a non-finite v in this value row, or kTc
  int any_bad[4];
  float red[4][kTc];  // squares of the outputs by TMEM lane quadrant
  float w[kTd];       // the norm's weights
  int abort;
  uint32_t tmem;
  // by chunk % 2, but gates by chunk % 4
  uint64_t full[2], empty[2], z[2], gates[4], p[2], k[2], o[2];
  uint64_t s, scores, outs, delta[2];
};

template <int MODE, bool CORE, bool GATED>
__global__ void __launch_bounds__(kPThreads, 1)
    decay_tc_kernel(const DecayArgs p, const DecaySegments sg, const __grid_constant__ CUtensorMap tm_q,
                      const __grid_constant__ CUtensorMap tm_k, const __grid_constant__ CUtensorMap tm_v,
                      const __grid_constant__ CUtensorMap tm_z, const __grid_constant__ CUtensorMap tm_o) {
  extern __shared__ __align__(1024) unsigned char smem_raw[];
  unsigned char* sm = smem_raw + ((1024u - (smem_u32(smem_raw) & 1023u)) & 1023u);
  __shared__ TcShared sh;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int slot = blockIdx.x / (unsigned)p.Hv;  // a segment's V heads side by side: they share q, k in L2
  const int h = blockIdx.x % (unsigned)p.Hv;
  const int kh = k_head_of(p.map, h, p.Hk, p.rep);
  DecaySegment s;
  if (!find_segment(p, sg, slot, lane, &s)) return;
  if (MODE == kPLocal && s.index + 1 == s.parts) return;
  const int chunks = (s.end - s.begin + kTc - 1) / kTc;

  if (warp == kPMma) {
    tc::tmem_alloc(&sh.tmem, kPCols);
    tc::tmem_relinquish();
  }
  if (tid == 0) {
    for (int i = 0; i < 2; ++i) {
      mbar_init(&sh.full[i], 1);
      mbar_init(&sh.empty[i], 1);
      mbar_init(&sh.z[i], 1);
      mbar_init(&sh.p[i], kPCompute);
      mbar_init(&sh.k[i], kPCompute);
      mbar_init(&sh.o[i], kPCompute);
      mbar_init(&sh.delta[i], 1);
    }
    for (int i = 0; i < 4; ++i) {
      mbar_init(&sh.gates[i], 1);
      sh.any_bad[i] = 0;
    }
    mbar_init(&sh.s, kPCompute);
    mbar_init(&sh.scores, 1);
    mbar_init(&sh.outs, 1);
    sh.abort = 0;
    fence_mbar_init();
  }
  if (tid < 4 * kTd) (&sh.bad[0][0])[tid] = kTc;
  if (GATED && tid < kTd) sh.w[tid] = p.norm_w[tid];
  tc::fence_before_sync();
  __syncthreads();
  tc::fence_after_sync();
  const uint32_t tb = sh.tmem;
  volatile int* abort_flag = &sh.abort;
  const auto wait = [&](uint64_t* bar, uint32_t parity) { return mbar_wait_bounded(bar, parity, abort_flag); };
  // the arrivals that give the last stages back are the MMA warp's last
  // commits: none may be under way when the CTA ends. For a warp that has seen
  // the phases before them (the load warp has, and the store warp with the
  // last o; the store warp's wait costs nothing: 93 us for one prompt, the
  // load warp's 98)
  const auto wait_given_back = [&]() {
    wait(&sh.empty[0], ((chunks + 1) / 2 - 1) & 1);
    if (chunks > 1) wait(&sh.empty[1], (chunks / 2 - 1) & 1);
  };
  const auto tokens = [&](int c) { return s.end - s.begin - c * kTc < kTc ? s.end - s.begin - c * kTc : kTc; };

  if (warp == kPMma) {
    // ---------------------------------------------------------------- MMAs
    const uint32_t id_s = tc::idesc(tc::kBF16, 64, 64), id_o1 = tc::idesc(tc::kBF16, 128, 64);
    const uint32_t id_o2 = id_o1 | kTransA, id_d = tc::idesc(tc::kBF16, 128, 128) | kTransA | kTransB;
    const uint64_t dP = tc::sdesc_sw128(smem_u32(sm + kPP));
    const auto all = [&](bool ok) { return __all_sync(0xffffffffu, ok); };
    const auto issue_scores = [&](int st) {
      const uint64_t dQ = tc::sdesc_sw128(smem_u32(sm + kPQ + st * kPTile));
      const uint64_t dK = tc::sdesc_sw128(smem_u32(sm + kPK + st * kPTile));
#pragma unroll
      for (int i = 0; i < 8; ++i)
        tc::mma_f16_elect(tb + kPColSc, tc::sdesc_at(dQ, 64, i), tc::sdesc_at(dK, 64, i), id_s, i > 0);
      tc::mma_commit_elect(&sh.scores);
    };
    const auto issue_o1 = [&](int st) {
      const uint64_t dQ = tc::sdesc_sw128(smem_u32(sm + kPQ + st * kPTile));
#pragma unroll
      for (int i = 0; i < 16; ++i)
        tc::mma_f16_ts_elect(tb + kPColO1, tb + kPColS + 8 * (i ^ 8), tc::sdesc_at(dQ, 64, i & 7), id_o1, i > 0);
    };
    bool ok = true;
    if (MODE == kPWhole) {
      ok = all(wait(&sh.full[0], 0));
      if (ok) issue_scores(0);
      ok = ok && all(wait(&sh.s, 0));
      tc::fence_after_sync();
      if (ok) issue_o1(0);
    }
    for (int c = 0; ok && c < chunks; ++c) {
      const int st = c & 1;
      const uint32_t round = (c >> 1) & 1;
      const uint64_t dV = sdesc_mn128(smem_u32(sm + kPV + st * kPTile));
      if (MODE == kPWhole) {
        ok = all(wait(&sh.p[st], round));
        if (!ok) break;
        tc::fence_after_sync();
#pragma unroll
        for (int i = 0; i < 8; ++i)
          tc::mma_f16_elect(tb + kPColO2, dV + ((i & 3) * 2048 >> 4), dP + (((1 - (i >> 2)) * 8192 + (i & 3) * 32) >> 4),
                            id_o2, i > 0);
        tc::mma_commit_elect(&sh.outs);
      }
      ok = all(wait(&sh.k[st], round));
      if (!ok) break;
      tc::fence_after_sync();
      const uint64_t dK0 = sdesc_mn128(smem_u32(sm + kPK + st * kPTile));
      const uint64_t dK1 = sdesc_mn128(smem_u32(sm + (MODE == kPLocal ? mid_at(st) : kPMid)));
      const uint32_t acc = tb + (MODE == kPLocal ? 128u * st : kPColKv);
#pragma unroll
      for (int i = 0; i < 12; ++i)
        tc::mma_f16_elect(acc, dV + ((i & 3) * 2048 >> 4),
                          (i < 4 ? dK1 + (kPTile >> 4) : i < 8 ? dK1 : dK0) + ((i & 3) * 2048 >> 4), id_d, i > 0);
      tc::mma_commit_elect(&sh.delta[MODE == kPLocal ? st : 0]);
      tc::mma_commit_elect(&sh.empty[st]);
      if (MODE == kPWhole && c + 1 < chunks) {
        ok = all(wait(&sh.full[st ^ 1], ((c + 1) >> 1) & 1));
        if (!ok) break;
        issue_scores(st ^ 1);
        ok = all(wait(&sh.s, (c + 1) & 1));
        if (!ok) break;
        tc::fence_after_sync();
        issue_o1(st ^ 1);
      }
    }
  } else if (warp == kPLoad) {
    // --------------------------------------------------------------- loads
    if (lane == 0) {
      const auto load = [&](int c) {
        const int st = c & 1, t0 = s.begin + c * kTc;
        mbar_arrive_expect_tx(&sh.full[st], (MODE == kPWhole ? 3 : 2) * kPTile);
        for (int b = 0; b < 2; ++b) {
          if (MODE == kPWhole)
            tc::tma_load_2d(sm + kPQ + st * kPTile + 8192 * b, &tm_q, kh * kTd + 64 * b, t0, &sh.full[st]);
          tc::tma_load_2d(sm + kPK + st * kPTile + 8192 * b, &tm_k, kh * kTd + 64 * b, t0, &sh.full[st]);
          tc::tma_load_2d(sm + kPV + st * kPTile + 8192 * b, &tm_v, h * kTd + 64 * b, t0, &sh.full[st]);
        }
      };
      load(0);
      int n = 1;
      for (; n < chunks; ++n) {
        if (n >= 2 && !wait(&sh.empty[n & 1], ((n >> 1) - 1) & 1)) break;
        load(n);
      }
      // none may be in flight when the CTA ends: load i went to stage i % 2
      mbar_wait(&sh.full[0], ((n + 1) / 2 - 1) & 1);
      if (n > 1) mbar_wait(&sh.full[1], (n / 2 - 1) & 1);
      if (MODE == kPLocal) wait_given_back();
    }
  } else if (warp == kPGates) {
    // ------------------------------------------------- sums of log decays
    // A buffer is written again four chunks later; o(c) seen means that every
    // warp has left chunk c - 1 (in the first pass: that the state has taken
    // chunk c). The compute warps cannot reach o(c + 2) before gates(c + 2),
    // given after o(c) was seen, so none is missed.
    float g0 = 0.f, g1 = 0.f;  // log decays of tokens 2 lane and 2 lane + 1 of a chunk
    const auto fetch_g = [&](int c) {
      const int64_t t = (int64_t)s.begin + c * kTc + 2 * lane;
      const float* g = p.g + t * p.g_stride + h;
      g0 = t < s.end ? g[0] : 0.f;
      g1 = t + 1 < s.end ? g[p.g_stride] : 0.f;
    };
    Two total{0.f, 0.f};  // of the segment, log2
    fetch_g(0);
    for (int c = 0; c < chunks; ++c) {
      if (MODE == kPWhole && c >= 2) __all_sync(0xffffffffu, wait(&sh.o[c & 1], ((c - 2) >> 1) & 1));
      if (MODE == kPLocal && c >= 3) __all_sync(0xffffffffu, wait(&sh.o[(c - 3) & 1], ((c - 3) >> 1) & 1));
      // inclusive sums over the chunk, as two floats; tokens past the chunk's
      // have log decay 0, so lane 31 ends with G_n
      const int at = c & 3, n = tokens(c);
      const Two first = to_log2(decay_log(g0));
      Two incl = add2(first, to_log2(decay_log(g1)));
      fetch_g(c + 1);
#pragma unroll
      for (int d = 1; d < 32; d <<= 1) {
        const Two o{__shfl_up_sync(0xffffffffu, incl.hi, d), __shfl_up_sync(0xffffffffu, incl.lo, d)};
        if (lane >= d) incl = add2(incl, o);
      }
      const Two prev{__shfl_up_sync(0xffffffffu, incl.hi, 1), __shfl_up_sync(0xffffffffu, incl.lo, 1)};
      const Two a = lane > 0 ? add2(prev, first) : first, b = incl;
      const Two gn{__shfl_sync(0xffffffffu, incl.hi, 31), __shfl_sync(0xffffffffu, incl.lo, 31)};
      if (MODE == kPWhole) {
        sh.G[at][2 * lane] = a;
        sh.G[at][2 * lane + 1] = b;
        sh.E[at][2 * lane] = p.scale * exp2_fast(a.hi + a.lo);
        sh.E[at][2 * lane + 1] = p.scale * exp2_fast(b.hi + b.lo);
        for (int i = lane; i < kTd; i += 32) sh.bad[at][i] = kTc;
        if (lane == 0) sh.any_bad[at] = 0;
      } else {
        total = add2(total, gn);
      }
      sh.dk[at][2 * lane] = 2 * lane < n ? exp2_fast((gn.hi - a.hi) + (gn.lo - a.lo)) : 0.f;
      sh.dk[at][2 * lane + 1] = 2 * lane + 1 < n ? exp2_fast((gn.hi - b.hi) + (gn.lo - b.lo)) : 0.f;
      if (lane == 0) sh.whole[at] = decay_factor((gn.hi + gn.lo) * kLn2);
      __syncwarp();
      if (lane == 0) mbar_arrive(&sh.gates[at]);
    }
    if (MODE == kPLocal && lane == 0 && !*abort_flag) sg.decays[(int64_t)(s.kept + s.index) * p.Hv + h] = exp2f(total.hi + total.lo);
  } else if (warp == kPStore) {
    // ------------------------------------------------------ z in, outputs out
    // (as for the gates: z(c + 2), or its place, is given after o(c) was seen)
    if (MODE == kPWhole) {
      uint32_t n_z = 0;
      const auto give_z = [&](int c) {
        const int st = c & 1;
        if (GATED) {
          ++n_z;
          mbar_arrive_expect_tx(&sh.z[st], kPTile);
          for (int b = 0; b < 2; ++b)
            tc::tma_load_2d(sm + kPO + st * kPTile + 8192 * b, &tm_z, h * kTd + 64 * b, s.begin + c * kTc, &sh.z[st]);
        } else {
          mbar_arrive(&sh.z[st]);
        }
      };
      if (lane == 0) {
        give_z(0);
        if (chunks > 1) give_z(1);
      }
      for (int c = 0; c < chunks; ++c) {
        const int st = c & 1;
        const bool ok = __all_sync(0xffffffffu, wait(&sh.o[st], (c >> 1) & 1));
        const int n = tokens(c), t0 = s.begin + c * kTc;
        const unsigned char* tile = sm + kPO + st * kPTile;
        if (ok && (!CORE || p.out != nullptr)) {
          if (n == kTc) {
            if (lane == 0) {
              for (int b = 0; b < 2; ++b) tc::tma_store_2d(&tm_o, h * kTd + 64 * b, t0, tile + 8192 * b);
              bulk_commit();
              bulk_wait_read_all();
            }
          } else {  // a last, shorter chunk: its rows alone
            for (int u = lane; u < 16 * n; u += 32) {
              const int t = u >> 4, c8 = u & 15;
              *reinterpret_cast<uint4*>(static_cast<__nv_bfloat16*>(p.out) + ((int64_t)(t0 + t) * p.Hv + h) * kTd + 8 * c8) =
                  *reinterpret_cast<const uint4*>(tile + (c8 >> 3) * 8192 + t * 128 + (((c8 & 7) ^ (t & 7)) << 4));
            }
          }
        }
        if (lane == 0 && c + 2 < chunks) give_z(c + 2);
      }
      if (lane == 0) {
        if (GATED) {
          mbar_wait(&sh.z[0], ((n_z + 1) / 2 - 1) & 1);
          if (n_z > 1) mbar_wait(&sh.z[1], (n_z / 2 - 1) & 1);
        }
        bulk_wait_all();
      }
      wait_given_back();
    }
  } else {
    // ------------------------------------------------------------- compute
    const int qd = warp & 3, hh = warp >> 2;
    const int j = 32 * qd + lane;  // this thread's value row; columns 32 hh .. 32 hh + 31 of the state
    const uint32_t tq = tb + ((uint32_t)(32 * qd) << 16);
    float2 S[16];
    float* gS = p.state + ((int64_t)s.seq * p.Hv + h) * (int64_t)(kTd * kTd);
    const int at0 = j * kTd + 32 * hh;
    {
      float4 x[8];
      if (MODE == kPLocal) {
#pragma unroll
        for (int e = 0; e < 8; ++e) x[e] = make_float4(0.f, 0.f, 0.f, 0.f);
        if (s.index == 0) {
          float* keep = sg.states + ((int64_t)(s.kept + s.parts - 1) * p.Hv + h) * (kTd * kTd);
#pragma unroll
          for (int e = 0; e < 4; ++e) load8(gS + at0 + 8 * e, x[2 * e], x[2 * e + 1]);
#pragma unroll
          for (int e = 0; e < 4; ++e) store8(keep + at0 + 8 * e, x[2 * e], x[2 * e + 1]);
        }
      } else if (s.parts == 1) {
#pragma unroll
        for (int e = 0; e < 4; ++e) load8(gS + at0 + 8 * e, x[2 * e], x[2 * e + 1]);
      } else {
        DecaySlots(p, sg, s, h, kTd * kTd).start8<4>(s.index, s.parts, at0, x);
      }
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        S[2 * e] = make_float2(x[e].x, x[e].y);
        S[2 * e + 1] = make_float2(x[e].z, x[e].w);
      }
    }
    bool failed = false;
    // all of the warp's tile is in place for the tensor cores or for TMA
    const auto hand = [&](uint64_t* bar) {
      fence_proxy_async_smem();
      tc::fence_before_sync();
      __syncwarp();
      if (lane == 0) mbar_arrive(bar);
    };
    // S as the A operand of O1: packed pairs, and what their rounding left
    const auto put_state = [&]() {
      uint32_t hi[16], lo[16];
#pragma unroll
      for (int e = 0; e < 16; ++e) {
        float2 a = S[e];
        hi[e] = split2(a);
        lo[e] = pack2(a);
      }
      tc::tmem_st16u(tq + kPColS + 64 + 16 * hh, lo);
      tc::tmem_st16u(tq + kPColS + 16 * hh, hi);
      tc::tmem_wait_st();
      hand(&sh.s);
    };
    // S <- e^(G_n) S + dS of chunk c
    const auto take_delta = [&](int c) {
      const Decay a = sh.whole[c & 3];
      const uint32_t parity = MODE == kPLocal ? (c >> 1) & 1 : c & 1;
      if (!wait(&sh.delta[MODE == kPLocal ? c & 1 : 0], parity)) failed = true;
      tc::fence_after_sync();
      float d[32];
      const uint32_t col = tq + (MODE == kPLocal ? 128u * (c & 1) : kPColKv) + 32 * hh;
      tc::tmem_ld16(col, *reinterpret_cast<float(*)[16]>(d));
      tc::tmem_ld16(col + 16, *reinterpret_cast<float(*)[16]>(d + 16));
      tc::tmem_wait_ld();
      const float2 f = make_float2(a.factor, a.factor), keep = make_float2(a.keep, a.keep);
      if (a.keep != 0.f) {
#pragma unroll
        for (int e = 0; e < 16; ++e) S[e] = fma2(f, S[e], fma2(keep, S[e], make_float2(d[2 * e], d[2 * e + 1])));
      } else {
#pragma unroll
        for (int e = 0; e < 16; ++e) S[e] = fma2(f, S[e], make_float2(d[2 * e], d[2 * e + 1]));
      }
      if (MODE == kPWhole && sh.any_bad[c & 3] && sh.bad[c & 3][j] < kTc)
#pragma unroll
        for (int e = 0; e < 16; ++e) S[e] = make_float2(__int_as_float(0x7fc00000), __int_as_float(0x7fc00000));
    };
    if (MODE == kPWhole) put_state();

    for (int c = 0; c < chunks; ++c) {
      const int n = tokens(c), st = c & 1, at = c & 3;
      const uint32_t round = (c >> 1) & 1;
      const Two* G = sh.G[at];
      if (!wait(&sh.gates[at], (c >> 2) & 1)) failed = true;
      if (!wait(&sh.full[st], round)) failed = true;
      unsigned char* kt = sm + kPK + st * kPTile;
      if (MODE == kPWhole) {
        // v: rows past the chunk's tokens are another sequence's (or stale): 0
        // there; non-finite elements are noted and replaced by 0
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          const int u = tid + i * 32 * kPCompute, row = u >> 4, c16 = u & 15;
          uint4* v = reinterpret_cast<uint4*>(sm + kPV + st * kPTile + (c16 >> 3) * 8192 + row * 128 +
                                              (((c16 & 7) ^ (row & 7)) << 4));
          uint4 x = *v;
          uint32_t* w = &x.x;
          uint32_t hit = 0;  // an exponent of all ones carries into the sign's place
#pragma unroll
          for (int e = 0; e < 4; ++e) hit |= (w[e] & 0x7f807f80u) + 0x00800080u;
          if (row >= n) {
            *v = make_uint4(0, 0, 0, 0);
          } else if ((hit & 0x80008000u) != 0) {
#pragma unroll
            for (int e = 0; e < 8; ++e)
              if (((w[e >> 1] >> (16 * (e & 1))) & 0x7f80u) == 0x7f80u) {
                atomicMin(&sh.bad[at][8 * c16 + e], row);
                w[e >> 1] &= e & 1 ? 0x0000ffffu : 0xffff0000u;
              }
            *v = x;
            sh.any_bad[at] = 1;
          }
        }
        // P: a lane has rows ta and ta + 8, columns s0 + 8 c and the next
        const int ta = 16 * qd + (lane >> 2), s0 = 16 * hh + 2 * (lane & 3);
        if (!wait(&sh.scores, c & 1)) failed = true;
        tc::fence_after_sync();
        float x[8];
        tmem_ld_16x16(tq + kPColSc + 16 * hh, x);
        tc::tmem_wait_ld();
        const Two ga = G[ta], gb = G[ta + 8];
        unsigned char* pp = sm + kPP + ta * 128 + 4 * (lane & 3);  // the rows are eight apart: the same swizzle
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          const int sc = s0 + 8 * i;
          const Two u0 = G[sc], u1 = G[sc + 1];
          float2 y = make_float2(x[4 * i] * exp2_fast((ga.hi - u0.hi) + (ga.lo - u0.lo)),
                                 x[4 * i + 1] * exp2_fast((ga.hi - u1.hi) + (ga.lo - u1.lo)));
          float2 z = make_float2(x[4 * i + 2] * exp2_fast((gb.hi - u0.hi) + (gb.lo - u0.lo)),
                                 x[4 * i + 3] * exp2_fast((gb.hi - u1.hi) + (gb.lo - u1.lo)));
          y = mul2(y, p.scale);
          z = mul2(z, p.scale);
          if (sc > ta) y.x = 0.f;
          if (sc + 1 > ta) y.y = 0.f;
          if (sc > ta + 8) z.x = 0.f;
          if (sc + 1 > ta + 8) z.y = 0.f;
          unsigned char* to = pp + (((2 * hh + i) ^ (ta & 7)) << 4);
          *reinterpret_cast<uint32_t*>(to) = split2(y);
          *reinterpret_cast<uint32_t*>(to + 1024) = split2(z);
          *reinterpret_cast<uint32_t*>(to + 8192) = pack2(y);
          *reinterpret_cast<uint32_t*>(to + 8192 + 1024) = pack2(z);
        }
        hand(&sh.p[st]);
      }

      // K' = e^(G_n - G_s) k in three parts, the first in place of K
      {
        unsigned char* mid = sm + (MODE == kPLocal ? mid_at(st) : kPMid);
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          const int u = tid + i * 32 * kPCompute, row = u >> 4, c16 = u & 15;
          const uint32_t off = (c16 >> 3) * 8192 + row * 128 + (((c16 & 7) ^ (row & 7)) << 4);
          uint4 x = *reinterpret_cast<const uint4*>(kt + off);
          if (row >= n) x = make_uint4(0, 0, 0, 0);  // another sequence's: may be a NaN
          const uint32_t* w = &x.x;
          const float d = sh.dk[at][row];
          uint4 part[3];
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            float2 a = mul2(unpack2(w[e]), d);
            (&part[0].x)[e] = cut2(a);
            (&part[1].x)[e] = cut2(a);
            (&part[2].x)[e] = __byte_perm(__float_as_uint(a.x), __float_as_uint(a.y), 0x7632);
          }
          *reinterpret_cast<uint4*>(kt + off) = part[0];
          *reinterpret_cast<uint4*>(mid + off) = part[1];
          *reinterpret_cast<uint4*>(mid + kPTile + off) = part[2];
        }
        hand(&sh.k[st]);
      }

      if (MODE == kPWhole) {
        if (!wait(&sh.z[st], round)) failed = true;
        if (!wait(&sh.outs, c & 1)) failed = true;
        tc::fence_after_sync();
        // o[a][2 c + b]: tokens tt + 8 c and the next, value row jj + 8 b + 16 a
        const int jj = 32 * qd + (lane >> 2), tt = 16 * hh + 2 * (lane & 3);
        float2 o[2][4];
        {
          float x[2][8], y[2][8];
#pragma unroll
          for (int a = 0; a < 2; ++a) {
            tmem_ld_16x16(tq + ((uint32_t)(16 * a) << 16) + kPColO1 + 16 * hh, x[a]);
            tmem_ld_16x16(tq + ((uint32_t)(16 * a) << 16) + kPColO2 + 16 * hh, y[a]);
          }
          tc::tmem_wait_ld();
#pragma unroll
          for (int i = 0; i < 2; ++i) {
            const float2 e = *reinterpret_cast<const float2*>(&sh.E[at][tt + 8 * i]);
#pragma unroll
            for (int a = 0; a < 2; ++a)
#pragma unroll
              for (int b = 0; b < 2; ++b)
                o[a][2 * i + b] = fma2(make_float2(x[a][4 * i + 2 * b], x[a][4 * i + 2 * b + 1]), e,
                                       make_float2(y[a][4 * i + 2 * b], y[a][4 * i + 2 * b + 1]));
          }
        }
        if (sh.any_bad[at])
#pragma unroll
          for (int i = 0; i < 8; ++i) {
            const int bad = sh.bad[at][jj + 16 * (i >> 2) + 8 * (i & 1)], t = tt + 8 * ((i >> 1) & 1);
            if (t >= bad) o[i >> 2][i & 3].x = __int_as_float(0x7fc00000);
            if (t + 1 >= bad) o[i >> 2][i & 3].y = __int_as_float(0x7fc00000);
          }
        if (CORE)
#pragma unroll
          for (int i = 0; i < 8; ++i) {
            const int t = tt + 8 * ((i >> 1) & 1);
            float* to = p.core_out + ((int64_t)(s.begin + c * kTc + t) * p.Hv + h) * kTd + jj + 16 * (i >> 2) + 8 * (i & 1);
            if (t < n) to[0] = o[i >> 2][i & 3].x;
            if (t + 1 < n) to[p.Hv * kTd] = o[i >> 2][i & 3].y;
          }
        float2 inv[2];
        if (GATED) {
          // squares over the value rows: the lanes' rows, then the four quadrants
#pragma unroll
          for (int i = 0; i < 2; ++i) {
            float2 sq = make_float2(0.f, 0.f);
#pragma unroll
            for (int a = 0; a < 2; ++a)
#pragma unroll
              for (int b = 0; b < 2; ++b) sq = fma2(o[a][2 * i + b], o[a][2 * i + b], sq);
#pragma unroll
            for (int d = 4; d < 32; d <<= 1) {
              sq.x += __shfl_xor_sync(0xffffffffu, sq.x, d);
              sq.y += __shfl_xor_sync(0xffffffffu, sq.y, d);
            }
            if (lane < 4) *reinterpret_cast<float2*>(&sh.red[qd][tt + 8 * i]) = sq;
          }
          // the four warps of these tokens; before the next chunk's squares
          // every one of them has read these (its outputs are handed on)
          asm volatile("bar.sync %0, 128;" ::"r"(1 + hh) : "memory");
#pragma unroll
          for (int i = 0; i < 2; ++i) {
            float2 r = make_float2(0.f, 0.f);
#pragma unroll
            for (int w = 0; w < 4; ++w) {
              const float2 x = *reinterpret_cast<const float2*>(&sh.red[w][tt + 8 * i]);
              r.x += x.x, r.y += x.y;
            }
            inv[i] = make_float2(rsqrtf(r.x * (1.f / kTd) + p.rms_eps), rsqrtf(r.y * (1.f / kTd) + p.rms_eps));
          }
        }
        // blocks (value rows b of half a) x (token blocks 0, 1)
#pragma unroll
        for (int a = 0; a < 2; ++a) {
          const int t = 16 * hh + 8 * (lane >> 4) + (lane & 7), c8 = 4 * qd + 2 * a + ((lane >> 3) & 1);
          const uint32_t to = smem_u32(sm + kPO + st * kPTile) + (c8 >> 3) * 8192 + t * 128 + (((c8 & 7) ^ (t & 7)) << 4);
          uint32_t r[4];
          if (GATED) {
            ldmatrix_t4(to, r);
            const float w0 = sh.w[jj + 16 * a], w1 = sh.w[jj + 16 * a + 8];
#pragma unroll
            for (int m = 0; m < 4; ++m) {
              const float2 z = unpack2(r[m]);
              const float2 e = mul2(z, -kLog2e);
              const float2 den = make_float2(1.f + exp2_fast(e.x), 1.f + exp2_fast(e.y));
              const float2 silu = make_float2(__fdividef(z.x, den.x), __fdividef(z.y, den.y));
              const float2 g = fma2(silu, mul2(inv[m >> 1], m & 1 ? w1 : w0), make_float2(-0.f, -0.f));
              o[a][m] = fma2(o[a][m], g, make_float2(-0.f, -0.f));
            }
          }
#pragma unroll
          for (int m = 0; m < 4; ++m) r[m] = pack2(o[a][m]);
          stmatrix_t4(to, r);
        }
        hand(&sh.o[st]);
        take_delta(c);
        if (c + 1 < chunks) put_state();
      } else if (c > 0) {
        take_delta(c - 1);
        hand(&sh.o[st ^ 1]);
      }
    }
    if (MODE == kPLocal) take_delta(chunks - 1);
    if (!failed && !*abort_flag && (MODE == kPLocal || s.index + 1 == s.parts)) {
      float* to = MODE == kPLocal ? sg.states + ((int64_t)(s.kept + s.index) * p.Hv + h) * (kTd * kTd) : gS;
#pragma unroll
      for (int e = 0; e < 4; ++e)
        store8(to + at0 + 8 * e, make_float4(S[4 * e].x, S[4 * e].y, S[4 * e + 1].x, S[4 * e + 1].y),
               make_float4(S[4 * e + 2].x, S[4 * e + 2].y, S[4 * e + 3].x, S[4 * e + 3].y));
    }
  }
  tc::fence_before_sync();
  __syncthreads();
  if (warp == kPMma) {
    tc::fence_after_sync();
    tc::tmem_dealloc(tb, kPCols);
  }
}

}  // namespace

bool decay_tc_fits(int32_t dtype, int32_t D, int32_t N, int64_t T) {
  // short sequences cost a CTA its start more than its chunk: up to 16 tokens
  // on average the scan is faster (64 sequences of 8 tokens, 32 heads: 82
  // against 131 us; of 16: 125 against 135; of 32: 219 against 142)
  return dtype == GDN_BF16 && D == kTd && T > 16ll * N;
}

bool decay_tc_supported(const DecayArgs& p) {
  // states are read and written in 32-byte accesses
  return reinterpret_cast<uintptr_t>(p.state) % 32 == 0 && tc::encode_fn() != nullptr;
}

cudaError_t launch_decay_tc(const DecayArgs& p, const DecaySegments& sg, cudaStream_t stream) {
  const CUtensorMapDataType bf = CU_TENSOR_MAP_DATA_TYPE_BFLOAT16;
  CUtensorMap mq, mk, mv, mz{}, mo{};  // the maps of what is not there are never used
  const int64_t vw = (int64_t)p.Hv * kTd;
  if (!tc::make_map_2d(&mq, p.q, p.T, (int64_t)p.Hk * kTd, p.q_stride, 2, bf, 64, kTc, CU_TENSOR_MAP_SWIZZLE_128B) ||
      !tc::make_map_2d(&mk, p.k, p.T, (int64_t)p.Hk * kTd, p.k_stride, 2, bf, 64, kTc, CU_TENSOR_MAP_SWIZZLE_128B) ||
      !tc::make_map_2d(&mv, p.v, p.T, vw, p.v_stride, 2, bf, 64, kTc, CU_TENSOR_MAP_SWIZZLE_128B) ||
      (p.z != nullptr && !tc::make_map_2d(&mz, p.z, p.T, vw, p.z_stride, 2, bf, 64, kTc, CU_TENSOR_MAP_SWIZZLE_128B)) ||
      (p.out != nullptr && !tc::make_map_2d(&mo, p.out, p.T, vw, vw, 2, bf, 64, kTc, CU_TENSOR_MAP_SWIZZLE_128B)))
    return cudaErrorInvalidValue;
  const unsigned grid = (unsigned)(sg.slots * p.Hv);
  const auto run = [&](auto* kernel) {
    constexpr int smem = (int)kPSmem + 1024;
    const cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
    if (e != cudaSuccess) return e;
    kernel<<<grid, kPThreads, smem, stream>>>(p, sg, mq, mk, mv, mz, mo);
    return cudaGetLastError();
  };
  if (sg.states != nullptr) {
    const cudaError_t e = run(decay_tc_kernel<kPLocal, false, false>);
    if (e != cudaSuccess) return e;
  }
  if (p.core_out != nullptr)
    return p.z != nullptr ? run(decay_tc_kernel<kPWhole, true, true>) : run(decay_tc_kernel<kPWhole, true, false>);
  return p.z != nullptr ? run(decay_tc_kernel<kPWhole, false, true>) : run(decay_tc_kernel<kPWhole, false, false>);
}

}  // namespace gdn

GDN_DEFINE_ERROR_READER(decay_tc)
