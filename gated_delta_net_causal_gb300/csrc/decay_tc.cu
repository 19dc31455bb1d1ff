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
// q, k and v are exact in bf16. Two parts leave 2^-17 of a factor, below what
// the 16-bit output keeps but visible in a state that is stored in fp32, so
// what is added to the state has three (2^-25).
//
// A CTA takes 96 KB of shared memory and 256 TMEM columns, so two share an SM
// and one's loads, exponentials and stores run under the other's products.
// Exponents are differences of sums of up to 64 log decays, which a decay of
// -100 a token makes large where the difference is small; the sums are held
// as two floats each.
//
// A NaN or an infinity in v times a masked P (0) would reach tokens before
// it: such elements of v are replaced by 0 before the product and make NaN in
// their value row of the outputs from their token on, and of the state.
//
// Segments (decay_common.cuh) run as in decay_scan.cu: a first pass adds up
// dS alone, the second starts each segment from what those before it leave.
#include <cuda.h>

#include "decay_common.cuh"
#include "tc_common.cuh"

namespace gdn {
namespace {

constexpr int kTc = 64;  // tokens per chunk
constexpr int kTd = 128;
constexpr int kTThreads = 256;
enum { kTWhole = 0, kTLocal = 1 };

// shared memory, from a 1024-byte boundary
constexpr uint32_t kOffQ = 0;        // [2 boxes of 64 columns][64 t][128 B] SW128
constexpr uint32_t kOffP = 16384;    // P hi, lo: [64 t][64 s] SW128 each
constexpr uint32_t kOffK = 32768;    // K, then K' hi in place
constexpr uint32_t kOffMid = 49152;  // K' mid
constexpr uint32_t kOffLo = 65536;   // K' lo
constexpr uint32_t kOffV = 81920;
constexpr uint32_t kTSmem = 98304;
constexpr uint32_t kTile16 = 16384;
// outputs [64 t][128 j] fp32 for the row pass, over Q and P once both are used
constexpr uint32_t kOffO = 0;

// TMEM columns
constexpr uint32_t kColS = 0;    // S hi (64 packed columns), S lo (64)
constexpr uint32_t kColX = 128;  // scores (64), then O2; dS (128) once O1 and O2 are read
constexpr uint32_t kColO1 = 192;
constexpr uint32_t kCols = 256;

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

// 16 lanes x 32 columns: thread lane holds rows lane/4 and lane/4 + 8,
// columns 8 c + 2 (lane % 4) and the next, at v[4 c], v[4 c + 1] and
// v[4 c + 2], v[4 c + 3]
__device__ __forceinline__ void tmem_ld_16x32(uint32_t taddr, float (&v)[16]) {
  uint32_t r[16];
  asm volatile(
      "tcgen05.ld.sync.aligned.16x256b.x4.b32 "
      "{%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15}, [%16];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]),
        "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
      : "r"(taddr));
#pragma unroll
  for (int i = 0; i < 16; ++i) v[i] = __uint_as_float(r[i]);
}

__device__ __forceinline__ float exp2_fast(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
// two floats to packed bf16 (a in the low half), and what the rounding left
__device__ __forceinline__ uint32_t split2(float& a, float& b) {
  uint32_t r;
  asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(b), "f"(a));
  a -= __uint_as_float(r << 16);
  b -= __uint_as_float(r & 0xffff0000u);
  return r;
}
__device__ __forceinline__ uint32_t pack2(float a, float b) {
  uint32_t r;
  asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(b), "f"(a));
  return r;
}

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

struct TcShared {
  Two G[kTc];       // sums of log2 decays
  float E[kTc];     // scale e^(G_t)
  float dk[kTc];    // e^(G_n - G_s), 0 past the chunk's tokens
  Decay whole;      // e^(G_n)
  int bad[kTd];     // first token of the chunk with a non-finite v in this value row, or kTc
  int any_bad;
  int abort;
  uint32_t tmem;
  uint64_t load, scores, outs, delta;  // mbarriers
};

template <int MODE>
__global__ void __launch_bounds__(kTThreads, 2)
    decay_tc_kernel(const DecayArgs p, const DecaySegments sg, const __grid_constant__ CUtensorMap tm_q,
                    const __grid_constant__ CUtensorMap tm_k, const __grid_constant__ CUtensorMap tm_v) {
  extern __shared__ __align__(1024) unsigned char smem_raw[];
  unsigned char* sm = smem_raw + ((1024u - (smem_u32(smem_raw) & 1023u)) & 1023u);
  __shared__ TcShared sh;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int qd = warp & 3, hh = warp >> 2;  // TMEM lane quadrant, column half
  const int j = 32 * qd + lane;             // this thread's value row
  const int64_t slot = blockIdx.x / (unsigned)p.Hv;  // a segment's V heads side by side: they share q, k in L2
  const int h = blockIdx.x % (unsigned)p.Hv;
  const int kh = k_head_of(p.map, h, p.Hk, p.rep);
  DecaySegment s;
  if (!find_segment(p, sg, slot, lane, &s)) return;
  if (MODE == kTLocal && s.index + 1 == s.parts) return;

  if (warp == 0) {
    tc::tmem_alloc(&sh.tmem, kCols);
    tc::tmem_relinquish();
  }
  if (tid == 0) {
    mbar_init(&sh.load, 1);
    mbar_init(&sh.scores, 1);
    mbar_init(&sh.outs, 1);
    mbar_init(&sh.delta, 1);
    sh.abort = 0;
    sh.any_bad = 0;
    fence_mbar_init();
  }
  if (tid < kTd) sh.bad[tid] = kTc;
  volatile int* abort_flag = &sh.abort;

  // the state: columns 64 hh .. 64 hh + 63 of row j
  float S[64];
  float* gS = p.state + ((int64_t)s.seq * p.Hv + h) * (int64_t)(kTd * kTd);
  const int at0 = j * kTd + 64 * hh;
  {
    const DecaySlots ws(p, sg, s, h, kTd * kTd);
    float* keep = sg.states + ((s.slot + s.parts - 1) * p.Hv + h) * (int64_t)(kTd * kTd);
#pragma unroll
    for (int c = 0; c < 16; ++c) {
      float4 x = make_float4(0.f, 0.f, 0.f, 0.f);
      if (MODE == kTLocal) {
        if (s.index == 0) {
          x = *reinterpret_cast<const float4*>(gS + at0 + 4 * c);
          *reinterpret_cast<float4*>(keep + at0 + 4 * c) = x;
        }
      } else {
        x = s.parts == 1 ? *reinterpret_cast<const float4*>(gS + at0 + 4 * c) : ws.start(s.index, s.parts, at0 + 4 * c);
      }
      S[4 * c] = x.x, S[4 * c + 1] = x.y, S[4 * c + 2] = x.z, S[4 * c + 3] = x.w;
    }
  }
  tc::fence_before_sync();
  __syncthreads();
  tc::fence_after_sync();
  const uint32_t tb = sh.tmem, tq = tb + ((uint32_t)(32 * qd) << 16);

  // S as the A operand of O1: packed pairs, hi then lo
  auto put_state = [&]() {
#pragma unroll
    for (int c = 0; c < 2; ++c) {
      uint32_t hi[16], lo[16];
#pragma unroll
      for (int e = 0; e < 16; ++e) {
        float a = S[32 * c + 2 * e], b = S[32 * c + 2 * e + 1];
        hi[e] = split2(a, b);
        lo[e] = pack2(a, b);
      }
      tc::tmem_st16u(tq + kColS + 32 * hh + 16 * c, hi);
      tc::tmem_st16u(tq + kColS + 64 + 32 * hh + 16 * c, lo);
    }
    tc::tmem_wait_st();
  };
  auto issue_loads = [&](int64_t t0) {
    mbar_arrive_expect_tx(&sh.load, (MODE == kTWhole ? 3 : 2) * kTile16);
#pragma unroll
    for (int b = 0; b < 2; ++b) {
      if (MODE == kTWhole) tc::tma_load_2d(sm + kOffQ + 8192 * b, &tm_q, kh * kTd + 64 * b, (int)t0, &sh.load);
      tc::tma_load_2d(sm + kOffK + 8192 * b, &tm_k, kh * kTd + 64 * b, (int)t0, &sh.load);
      tc::tma_load_2d(sm + kOffV + 8192 * b, &tm_v, h * kTd + 64 * b, (int)t0, &sh.load);
    }
  };
  // log decays of tokens 2 lane and 2 lane + 1 of a chunk (warp 1)
  float g0 = 0.f, g1 = 0.f;
  auto fetch_g = [&](int64_t t0) {
    const int64_t t = t0 + 2 * lane;
    g0 = t < s.end ? decay_log(p.g[t * p.g_stride + h]) : 0.f;
    g1 = t + 1 < s.end ? decay_log(p.g[(t + 1) * p.g_stride + h]) : 0.f;
  };

  if (MODE == kTWhole) put_state();
  if (tid == 0) issue_loads(s.begin);
  if (warp == 1) fetch_g(s.begin);
  Two total{0.f, 0.f};  // of the segment, log2
  uint32_t loads = 1;
  const uint32_t aQ = smem_u32(sm + kOffQ), aP = smem_u32(sm + kOffP);
  const uint64_t dQ = tc::sdesc_sw128(aQ), dK = tc::sdesc_sw128(smem_u32(sm + kOffK)), dP = tc::sdesc_sw128(aP);
  const uint64_t dV = sdesc_mn128(smem_u32(sm + kOffV)), dKp = sdesc_mn128(smem_u32(sm + kOffK));
  bool failed = false;
  uint32_t phase = 0;
  // #1: the state operand is in TMEM and the buffers are free
  tc::fence_before_sync();
  __syncthreads();

  for (int64_t t0 = s.begin; t0 < s.end; t0 += kTc, phase ^= 1) {
    const int n = s.end - t0 < kTc ? (int)(s.end - t0) : kTc;
    if (!mbar_wait_bounded(&sh.load, phase, abort_flag)) failed = true;
    if (MODE == kTWhole && warp == 0) {
      tc::fence_after_sync();
      const uint32_t id_s = tc::idesc(tc::kBF16, 64, 64), id_o = tc::idesc(tc::kBF16, 128, 64);
#pragma unroll
      for (int k = 0; k < 8; ++k)
        tc::mma_f16_elect(tb + kColX, tc::sdesc_at(dQ, 64, k), tc::sdesc_at(dK, 64, k), id_s, k > 0);
      tc::mma_commit_elect(&sh.scores);
#pragma unroll
      for (int k = 0; k < 16; ++k)
        tc::mma_f16_ts_elect(tb + kColO1, tb + kColS + 8 * k, tc::sdesc_at(dQ, 64, k & 7), id_o, k > 0);
    }
    if (warp == 1) {
      // inclusive sums over the chunk, as two floats
      const Two first = to_log2(g0);
      Two incl = add2(first, to_log2(g1));
#pragma unroll
      for (int d = 1; d < 32; d <<= 1) {
        const Two o{__shfl_up_sync(0xffffffffu, incl.hi, d), __shfl_up_sync(0xffffffffu, incl.lo, d)};
        if (lane >= d) incl = add2(incl, o);
      }
      const Two prev{__shfl_up_sync(0xffffffffu, incl.hi, 1), __shfl_up_sync(0xffffffffu, incl.lo, 1)};
      const Two a = lane > 0 ? add2(prev, first) : first, b = incl;
      // tokens past the chunk's have log decay 0, so lane 31 holds G_n
      const Two gn{__shfl_sync(0xffffffffu, incl.hi, 31), __shfl_sync(0xffffffffu, incl.lo, 31)};
      if (MODE == kTWhole) {
        sh.G[2 * lane] = a;
        sh.G[2 * lane + 1] = b;
        sh.E[2 * lane] = p.scale * exp2_fast(a.hi + a.lo);
        sh.E[2 * lane + 1] = p.scale * exp2_fast(b.hi + b.lo);
      } else {
        total = add2(total, gn);
      }
      sh.dk[2 * lane] = 2 * lane < n ? exp2_fast((gn.hi - a.hi) + (gn.lo - a.lo)) : 0.f;
      sh.dk[2 * lane + 1] = 2 * lane + 1 < n ? exp2_fast((gn.hi - b.hi) + (gn.lo - b.lo)) : 0.f;
      if (lane == 0) sh.whole = decay_factor((gn.hi + gn.lo) * kLn2);
      if (t0 + kTc < s.end) fetch_g(t0 + kTc);
    }
    // v: rows past the chunk's tokens are another sequence's (or stale): 0
    // there; non-finite elements are noted and replaced by 0
    if (MODE == kTWhole || n < kTc) {
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int u = tid + i * kTThreads, row = u >> 4, c16 = u & 15;
        uint4* at = reinterpret_cast<uint4*>(sm + kOffV + (c16 >> 3) * 8192 + row * 128 + (((c16 & 7) ^ (row & 7)) << 4));
        if (row >= n) {
          *at = make_uint4(0, 0, 0, 0);
        } else if (MODE == kTWhole) {
          uint4 x = *at;
          uint32_t* w = &x.x;
          uint32_t hit = 0;
#pragma unroll
          for (int e = 0; e < 4; ++e) hit |= __vcmpeq2(w[e] & 0x7f807f80u, 0x7f807f80u);
          if (hit != 0) {
#pragma unroll
            for (int e = 0; e < 8; ++e)
              if (((w[e >> 1] >> (16 * (e & 1))) & 0x7f80u) == 0x7f80u) {
                atomicMin(&sh.bad[8 * c16 + e], row);
                w[e >> 1] &= e & 1 ? 0x0000ffffu : 0xffff0000u;
              }
            *at = x;
            sh.any_bad = 1;
          }
        }
      }
    }
    __syncthreads();  // #2: the sums are in shared memory

    if (MODE == kTWhole) {
      if (!mbar_wait_bounded(&sh.scores, phase, abort_flag)) failed = true;
      tc::fence_after_sync();
      float x[16];
      tmem_ld_16x32(tq + kColX + 32 * hh, x);
      tc::tmem_wait_ld();
      const int ta = 16 * qd + (lane >> 2), tb2 = ta + 8, s0 = 32 * hh + 2 * (lane & 3);
      const Two ga = sh.G[ta], gb = sh.G[tb2];
#pragma unroll
      for (int c = 0; c < 4; ++c) {
        const int sc = s0 + 8 * c;
        const Two u0 = sh.G[sc], u1 = sh.G[sc + 1];
        float y[4];
        y[0] = sc <= ta ? x[4 * c] * p.scale * exp2_fast((ga.hi - u0.hi) + (ga.lo - u0.lo)) : 0.f;
        y[1] = sc + 1 <= ta ? x[4 * c + 1] * p.scale * exp2_fast((ga.hi - u1.hi) + (ga.lo - u1.lo)) : 0.f;
        y[2] = sc <= tb2 ? x[4 * c + 2] * p.scale * exp2_fast((gb.hi - u0.hi) + (gb.lo - u0.lo)) : 0.f;
        y[3] = sc + 1 <= tb2 ? x[4 * c + 3] * p.scale * exp2_fast((gb.hi - u1.hi) + (gb.lo - u1.lo)) : 0.f;
        // rows ta and tb2 are eight apart: the same swizzle
        const uint32_t off = ta * 128 + (((4 * hh + c) ^ (ta & 7)) << 4) + 4 * (lane & 3);
        *reinterpret_cast<uint32_t*>(sm + kOffP + off) = split2(y[0], y[1]);
        *reinterpret_cast<uint32_t*>(sm + kOffP + 8192 + off) = pack2(y[0], y[1]);
        *reinterpret_cast<uint32_t*>(sm + kOffP + off + 1024) = split2(y[2], y[3]);
        *reinterpret_cast<uint32_t*>(sm + kOffP + 8192 + off + 1024) = pack2(y[2], y[3]);
      }
      fence_proxy_async_smem();
      tc::fence_before_sync();
      __syncthreads();  // #3: P and v are in shared memory, the scores are read
      if (warp == 0) {
        tc::fence_after_sync();
        const uint32_t id = tc::idesc(tc::kBF16, 128, 64) | kTransA;
#pragma unroll
        for (int k = 0; k < 8; ++k)
          tc::mma_f16_elect(tb + kColX, dV + ((k & 3) * 2048 >> 4),
                            dP + (((k >> 2) * 8192 + (k & 3) * 32) >> 4), id, k > 0);
        tc::mma_commit_elect(&sh.outs);
      }
    }

    // K' = e^(G_n - G_s) k in three parts, the first in place of K
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int u = tid + i * kTThreads, row = u >> 4, c16 = u & 15;
      const uint32_t off = (c16 >> 3) * 8192 + row * 128 + (((c16 & 7) ^ (row & 7)) << 4);
      const uint4 x = *reinterpret_cast<const uint4*>(sm + kOffK + off);
      const uint32_t* w = &x.x;
      const float d = sh.dk[row];
      uint4 part[3];
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        float a = __uint_as_float(w[e] << 16) * d, b = __uint_as_float(w[e] & 0xffff0000u) * d;
        if (row >= n) a = b = 0.f;  // not a product: the row may hold a NaN
        (&part[0].x)[e] = split2(a, b);
        (&part[1].x)[e] = split2(a, b);
        (&part[2].x)[e] = pack2(a, b);
      }
      *reinterpret_cast<uint4*>(sm + kOffK + off) = part[0];
      *reinterpret_cast<uint4*>(sm + kOffMid + off) = part[1];
      *reinterpret_cast<uint4*>(sm + kOffLo + off) = part[2];
    }
    fence_proxy_async_smem();

    if (MODE == kTWhole) {
      if (!mbar_wait_bounded(&sh.outs, phase, abort_flag)) failed = true;
      tc::fence_after_sync();
      const int bad = sh.any_bad ? sh.bad[j] : kTc;
#pragma unroll
      for (int c = 0; c < 2; ++c) {
        float a[16], b[16];
        tc::tmem_ld16(tq + kColO1 + 32 * hh + 16 * c, a);
        tc::tmem_ld16(tq + kColX + 32 * hh + 16 * c, b);
        tc::tmem_wait_ld();
#pragma unroll
        for (int e = 0; e < 16; ++e) {
          const int t = 32 * hh + 16 * c + e;
          float o = fmaf(a[e], sh.E[t], b[e]);
          if (t >= bad) o = __int_as_float(0x7fc00000);
          *reinterpret_cast<float*>(sm + kOffO + (t * kTd + j) * 4) = o;
        }
      }
    }
    tc::fence_before_sync();
    __syncthreads();  // #4: K' is in shared memory, the outputs are staged and their TMEM columns read
    if (warp == 0) {
      tc::fence_after_sync();
      const uint32_t id = tc::idesc(tc::kBF16, 128, 128) | kTransA | kTransB;
#pragma unroll
      for (int k = 0; k < 12; ++k)
        tc::mma_f16_elect(tb + kColX, dV + ((k & 3) * 2048 >> 4), dKp + (((k >> 2) * kTile16 + (k & 3) * 2048) >> 4), id,
                          k > 0);
      tc::mma_commit_elect(&sh.delta);
    }
    if (MODE == kTWhole) {
      // rows of the outputs: eight tokens a warp, four value rows a lane
      const __nv_bfloat16* z = static_cast<const __nv_bfloat16*>(p.z);
      float4 w4 = make_float4(0.f, 0.f, 0.f, 0.f);
      if (z != nullptr) w4 = *reinterpret_cast<const float4*>(p.norm_w + 4 * lane);
#pragma unroll 4
      for (int r = 0; r < 8; ++r) {
        const int t = 8 * warp + r;
        if (t >= n) break;
        const int64_t orow = ((t0 + t) * p.Hv + h) * kTd + 4 * lane;
        float4 o = *reinterpret_cast<const float4*>(sm + kOffO + (t * kTd + 4 * lane) * 4);
        if (p.core_out != nullptr) *reinterpret_cast<float4*>(p.core_out + orow) = o;
        if (z != nullptr) {
          const float4 zz = load4(z + (t0 + t) * p.z_stride + h * kTd + 4 * lane);
          const float ss = group_sum<32>(o.x * o.x + o.y * o.y + (o.z * o.z + o.w * o.w));
          const float inv = 1.f / sqrtf(ss * (1.f / kTd) + p.rms_eps);
          o = make_float4(o.x * inv * w4.x * silu_fast(zz.x), o.y * inv * w4.y * silu_fast(zz.y),
                          o.z * inv * w4.z * silu_fast(zz.z), o.w * inv * w4.w * silu_fast(zz.w));
        }
        if (p.out != nullptr)
          *reinterpret_cast<uint2*>(static_cast<__nv_bfloat16*>(p.out) + orow) =
              make_uint2(pack2(o.x, o.y), pack2(o.z, o.w));
      }
    }
    if (!mbar_wait_bounded(&sh.delta, phase, abort_flag)) failed = true;
    tc::fence_after_sync();
    {
      const Decay a = sh.whole;
      const bool spoilt = MODE == kTWhole && sh.any_bad && sh.bad[j] < kTc;
#pragma unroll
      for (int c = 0; c < 4; ++c) {
        float d[16];
        tc::tmem_ld16(tq + kColX + 64 * hh + 16 * c, d);
        tc::tmem_wait_ld();
#pragma unroll
        for (int e = 0; e < 16; ++e) {
          S[16 * c + e] = fmaf(a.factor, S[16 * c + e], a.keep != 0.f ? S[16 * c + e] + d[e] : d[e]);
          if (spoilt) S[16 * c + e] = __int_as_float(0x7fc00000);
        }
      }
      if (MODE == kTWhole) put_state();
    }
    fence_proxy_async_smem();
    tc::fence_before_sync();
    // #1 of the next chunk: everything of this one is read
    if (__syncthreads_or(failed)) break;
    if (MODE == kTWhole && sh.any_bad) {
      __syncthreads();
      if (tid < kTd) sh.bad[tid] = kTc;
      if (tid == 0) sh.any_bad = 0;
      __syncthreads();
    }
    if (t0 + kTc < s.end && tid == 0) {
      issue_loads(t0 + kTc);
      ++loads;
    }
  }

  if (!failed && !*abort_flag) {
    if (MODE == kTLocal || s.index + 1 == s.parts) {
      float* to = MODE == kTLocal ? sg.states + (int64_t)blockIdx.x * (kTd * kTd) : gS;
#pragma unroll
      for (int c = 0; c < 16; ++c)
        *reinterpret_cast<float4*>(to + at0 + 4 * c) =
            make_float4(S[4 * c], S[4 * c + 1], S[4 * c + 2], S[4 * c + 3]);
    }
    if (MODE == kTLocal && warp == 1 && lane == 0) sg.decays[blockIdx.x] = exp2f(total.hi + total.lo);
  }
  // no load may still be in flight when the CTA ends
  if (tid == 0) mbar_wait(&sh.load, (loads - 1) & 1);
  tc::fence_before_sync();
  __syncthreads();
  if (warp == 0) {
    tc::fence_after_sync();
    tc::tmem_dealloc(tb, kCols);
  }
}

}  // namespace

bool decay_tc_supported(const DecayArgs&, int32_t dtype, int32_t D) {
  return dtype == GDN_BF16 && D == kTd && tc::encode_fn() != nullptr;
}

cudaError_t launch_decay_tc(const DecayArgs& p, const DecaySegments& sg, cudaStream_t stream) {
  const CUtensorMapDataType bf = CU_TENSOR_MAP_DATA_TYPE_BFLOAT16;
  CUtensorMap mq, mk, mv;
  if (!tc::make_map_2d(&mq, p.q, p.T, (int64_t)p.Hk * kTd, p.q_stride, 2, bf, 64, kTc, CU_TENSOR_MAP_SWIZZLE_128B) ||
      !tc::make_map_2d(&mk, p.k, p.T, (int64_t)p.Hk * kTd, p.k_stride, 2, bf, 64, kTc, CU_TENSOR_MAP_SWIZZLE_128B) ||
      !tc::make_map_2d(&mv, p.v, p.T, (int64_t)p.Hv * kTd, p.v_stride, 2, bf, 64, kTc, CU_TENSOR_MAP_SWIZZLE_128B))
    return cudaErrorInvalidValue;
  const unsigned grid = (unsigned)(sg.slots * p.Hv);
  constexpr int smem = (int)kTSmem + 1024;
  auto whole = decay_tc_kernel<kTWhole>;
  auto local = decay_tc_kernel<kTLocal>;
  cudaError_t e = cudaFuncSetAttribute(whole, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
  if (e == cudaSuccess) e = cudaFuncSetAttribute(local, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
  if (e != cudaSuccess) return e;
  if (sg.states != nullptr) {
    local<<<grid, kTThreads, smem, stream>>>(p, sg, mq, mk, mv);
    e = cudaGetLastError();
    if (e != cudaSuccess) return e;
  }
  whole<<<grid, kTThreads, smem, stream>>>(p, sg, mq, mk, mv);
  return cudaGetLastError();
}

}  // namespace gdn

GDN_DEFINE_ERROR_READER(decay_tc)
