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
//   O1      [j][t] = S Q^T               S from TMEM, rounded to bf16
//   O2      [j][t] = V^T P^T             V read transposed, P rounded to bf16
//   dS      [j][i] = V^T K'              K' = e^(G_n - G_s) k as bf16 hi + mid + lo
// q, k and v are exact in bf16. What is added to the state has three bf16
// parts (2^-24 of a factor), as the state is kept in fp32. S and P only reach
// the outputs: one part each where out alone is asked for, whose own rounding
// is as large (together 1.4 times it), two (2^-17) where core_out is.
//
// An MMA of these sizes holds the tensor pipe for about 73 cycles whatever
// its M and N, so what counts is their number: 32 a chunk (44 with core_out).
// A CTA takes 104 KB of shared memory and 256 TMEM columns, so two share an SM
// and one's loads, exponentials and stores run under the other's products.
// The outputs leave TMEM as 8 x 8 blocks, are normed and gated in registers
// (z comes by TMA as they go, transposed in shared memory) and whole chunks
// are stored by TMA while dS is computed.
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
#include "decay_tc.cuh"

namespace gdn {
namespace {

constexpr int kTThreads = 256;
constexpr int kGateWarp = 1, kStoreWarp = 2, kDeltaWarp = 6;
enum { kTWhole = 0, kTLocal = 1 };

// shared memory, from a 1024-byte boundary; tiles of 64 tokens x 128 columns
// are two boxes of 64 columns, 128-byte swizzled rows
constexpr uint32_t kOffQ = 0;
constexpr uint32_t kOffK = 16384;    // K, then K' hi in place
constexpr uint32_t kOffMid = 32768;  // K' mid
constexpr uint32_t kOffLo = 49152;   // K' lo
constexpr uint32_t kOffV = 65536;
constexpr uint32_t kOffO = 81920;    // z, then the outputs in its place
constexpr uint32_t kOffP = 98304;    // P [64 t][64 s] SW128, with core_out its low part behind it
constexpr uint32_t kTile16 = 16384;
// the first pass has no q, P or outputs: their place is a second stage of K and V
__device__ __forceinline__ uint32_t k_at(int stage) { return stage ? kOffO : kOffK; }
__device__ __forceinline__ uint32_t v_at(int stage) { return stage ? kOffQ : kOffV; }
constexpr uint32_t tc_smem(bool core) { return kOffP + (core ? 16384 : 8192); }

// TMEM columns
constexpr uint32_t kColS = 0;    // S hi (64 packed columns), S lo (64)
constexpr uint32_t kColX = 128;  // scores (64), then O2; dS (128) once O1 and O2 are read
constexpr uint32_t kColO1 = 192;
constexpr uint32_t kCols = 256;

struct TcShared {
  Two G[2][kTc];    // sums of a chunk's log2 decays, by chunk parity
  float E[kTc];     // scale e^(G_t)
  float dk[kTc];    // e^(G_n - G_s), 0 past the chunk's tokens
  float w[kTd];       // the norm's weights
  float red[4][kTc];  // squares of the outputs by TMEM lane quadrant
  int bad[2][kTd];  // by chunk parity: first token with a non-finite v in this value row, or kTc
  int any_bad[2];
  int abort;
  uint32_t tmem;
  uint64_t load_q, load_kv[2], load_z, scores, outs, delta;  // mbarriers
};

template <int MODE, bool CORE, bool GATED>
__global__ void __launch_bounds__(kTThreads, 2)
    decay_tc_kernel(const DecayArgs p, const DecaySegments sg, const __grid_constant__ CUtensorMap tm_q,
                    const __grid_constant__ CUtensorMap tm_k, const __grid_constant__ CUtensorMap tm_v,
                    const __grid_constant__ CUtensorMap tm_z, const __grid_constant__ CUtensorMap tm_o) {
  extern __shared__ __align__(1024) unsigned char smem_raw[];
  unsigned char* sm = smem_raw + ((1024u - (smem_u32(smem_raw) & 1023u)) & 1023u);
  __shared__ TcShared sh;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int qd = warp & 3, hh = warp >> 2;  // TMEM lane quadrant, column half
  const int j = 32 * qd + lane;             // this thread's value row
  const int slot = blockIdx.x / (unsigned)p.Hv;  // a segment's V heads side by side: they share q, k in L2
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
    mbar_init(&sh.load_q, 1);
    mbar_init(&sh.load_kv[0], 1);
    mbar_init(&sh.load_kv[1], 1);
    mbar_init(&sh.load_z, 1);
    mbar_init(&sh.scores, 1);
    mbar_init(&sh.outs, 2);  // O1 and O2
    mbar_init(&sh.delta, 1);
    sh.abort = 0;
    sh.any_bad[0] = sh.any_bad[1] = 0;
    fence_mbar_init();
  }
  if (tid < 2 * kTd) (&sh.bad[0][0])[tid] = kTc;
  if (GATED && tid < kTd) sh.w[tid] = p.norm_w[tid];
  volatile int* abort_flag = &sh.abort;

  // the state: columns 64 hh .. 64 hh + 63 of row j
  float2 S[32];
  float* gS = p.state + ((int64_t)s.seq * p.Hv + h) * (int64_t)(kTd * kTd);
  const int at0 = j * kTd + 64 * hh;
  {
    const DecaySlots ws(p, sg, s, h, kTd * kTd);
    float* keep = sg.states + ((int64_t)(s.slot + s.parts - 1) * p.Hv + h) * (kTd * kTd);
#pragma unroll
    for (int c = 0; c < 2; ++c) {
      float4 x[8];
      if (MODE == kTLocal) {
#pragma unroll
        for (int e = 0; e < 8; ++e) x[e] = make_float4(0.f, 0.f, 0.f, 0.f);
        if (s.index == 0) {
#pragma unroll
          for (int e = 0; e < 4; ++e) load8(gS + at0 + 32 * c + 8 * e, x[2 * e], x[2 * e + 1]);
#pragma unroll
          for (int e = 0; e < 4; ++e) store8(keep + at0 + 32 * c + 8 * e, x[2 * e], x[2 * e + 1]);
        }
      } else if (s.parts == 1) {
#pragma unroll
        for (int e = 0; e < 4; ++e) load8(gS + at0 + 32 * c + 8 * e, x[2 * e], x[2 * e + 1]);
      } else {
        ws.start8<4>(s.index, s.parts, at0 + 32 * c, x);
      }
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        S[16 * c + 2 * e] = make_float2(x[e].x, x[e].y);
        S[16 * c + 2 * e + 1] = make_float2(x[e].z, x[e].w);
      }
    }
  }
  tc::fence_before_sync();
  __syncthreads();
  tc::fence_after_sync();
  const uint32_t tb = sh.tmem, tq = tb + ((uint32_t)(32 * qd) << 16);

  // columns 64 hh + 32 c .. + 31 of S as the A operand of O1: packed pairs,
  // and with core_out what their rounding left
  auto put_state = [&](int c) {
    uint32_t hi[16];
    if (CORE) {
      uint32_t lo[16];
#pragma unroll
      for (int e = 0; e < 16; ++e) {
        float2 a = S[16 * c + e];
        hi[e] = split2(a);
        lo[e] = pack2(a);
      }
      tc::tmem_st16u(tq + kColS + 64 + 32 * hh + 16 * c, lo);
    } else {
#pragma unroll
      for (int e = 0; e < 16; ++e) hi[e] = pack2(S[16 * c + e]);
    }
    tc::tmem_st16u(tq + kColS + 32 * hh + 16 * c, hi);
  };
  uint32_t q_loads = 0, kv_loads = 0, z_loads = 0;  // thread 0's, z the store warp's lane 0's
  auto load_q = [&](int t0) {
    ++q_loads;
    mbar_arrive_expect_tx(&sh.load_q, kTile16);
    for (int b = 0; b < 2; ++b) tc::tma_load_2d(sm + kOffQ + 8192 * b, &tm_q, kh * kTd + 64 * b, t0, &sh.load_q);
  };
  auto load_kv = [&](int t0, int stage) {
    ++kv_loads;
    mbar_arrive_expect_tx(&sh.load_kv[stage], 2 * kTile16);
    for (int b = 0; b < 2; ++b) {
      tc::tma_load_2d(sm + k_at(stage) + 8192 * b, &tm_k, kh * kTd + 64 * b, t0, &sh.load_kv[stage]);
      tc::tma_load_2d(sm + v_at(stage) + 8192 * b, &tm_v, h * kTd + 64 * b, t0, &sh.load_kv[stage]);
    }
  };
  auto load_z = [&](int t0) {
    ++z_loads;
    mbar_arrive_expect_tx(&sh.load_z, kTile16);
    for (int b = 0; b < 2; ++b) tc::tma_load_2d(sm + kOffO + 8192 * b, &tm_z, h * kTd + 64 * b, t0, &sh.load_z);
  };
  // log decays of tokens 2 lane and 2 lane + 1 of a chunk, and its gates (warp 1)
  float g0 = 0.f, g1 = 0.f;
  Two total{0.f, 0.f}, gn{0.f, 0.f};  // log2, of the segment and the chunk
  auto fetch_g = [&](int t0) {
    const int t = t0 + 2 * lane;
    const float* g = p.g + t * p.g_stride + h;
    g0 = t < s.end ? g[0] : 0.f;
    g1 = t + 1 < s.end ? g[p.g_stride] : 0.f;
  };
  auto put_sums = [&](Two* to) {
    // inclusive sums over the chunk, as two floats; tokens past the chunk's
    // have log decay 0, so lane 31 ends with G_n
    const Two first = to_log2(decay_log(g0));
    Two incl = add2(first, to_log2(decay_log(g1)));
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
      const Two o{__shfl_up_sync(0xffffffffu, incl.hi, d), __shfl_up_sync(0xffffffffu, incl.lo, d)};
      if (lane >= d) incl = add2(incl, o);
    }
    const Two prev{__shfl_up_sync(0xffffffffu, incl.hi, 1), __shfl_up_sync(0xffffffffu, incl.lo, 1)};
    to[2 * lane] = lane > 0 ? add2(prev, first) : first;
    to[2 * lane + 1] = incl;
    if (MODE == kTLocal) gn = Two{__shfl_sync(0xffffffffu, incl.hi, 31), __shfl_sync(0xffffffffu, incl.lo, 31)};
  };
  const auto tokens = [&](int t0) { return s.end - t0 < kTc ? s.end - t0 : kTc; };

  if (tid == 0) {
    load_kv(s.begin, 0);
    if (MODE == kTLocal && s.begin + kTc < s.end) load_kv(s.begin + kTc, 1);
    if (MODE == kTWhole) load_q(s.begin);
  }
  if (GATED && warp == kStoreWarp && lane == 0) load_z(s.begin);
  if (warp == 1) {
    fetch_g(s.begin);
    put_sums(sh.G[0]);
    total = gn;
    fetch_g(s.begin + kTc);
  }
  if (MODE == kTWhole) {
    put_state(0);
    put_state(1);
    tc::tmem_wait_st();
  }
  const uint64_t dQ = tc::sdesc_sw128(smem_u32(sm + kOffQ)), dK = tc::sdesc_sw128(smem_u32(sm + kOffK));
  const uint64_t dP = tc::sdesc_sw128(smem_u32(sm + kOffP));
  const uint64_t dMid = sdesc_mn128(smem_u32(sm + kOffMid));
  bool failed = false;
  uint32_t phase = 0, round = 0;  // parities of the chunk and, in the first pass, of its stage
  // #1: the state operand is in TMEM, the gates in shared memory
  tc::fence_before_sync();
  __syncthreads();

  for (int t0 = s.begin; t0 < s.end; t0 += kTc, phase ^= 1, round ^= phase ^ 1) {
    const int n = tokens(t0);
    const bool more = t0 + kTc < s.end;
    const Two* G = sh.G[phase];
    const int stage = MODE == kTLocal ? (int)phase : 0;
    unsigned char *kt = sm + k_at(stage), *vt = sm + v_at(stage);
    const uint64_t dV = sdesc_mn128(smem_u32(vt));
    // the buffers are single: the next chunk's tiles come into L2 meanwhile, so
    // that its loads, issued late in this chunk, are short
    if (MODE == kTWhole && warp == 7 && lane == 0 && more) {
      for (int b = 0; b < 2; ++b) {
        tc::tma_prefetch_2d(&tm_k, kh * kTd + 64 * b, t0 + kTc);
        tc::tma_prefetch_2d(&tm_v, h * kTd + 64 * b, t0 + kTc);
        tc::tma_prefetch_2d(&tm_q, kh * kTd + 64 * b, t0 + kTc);
        if (GATED) tc::tma_prefetch_2d(&tm_z, h * kTd + 64 * b, t0 + kTc);
      }
    }
    if (!mbar_wait_bounded(&sh.load_kv[stage], MODE == kTLocal ? round : phase, abort_flag)) failed = true;
    if (MODE == kTWhole) {
      if (!mbar_wait_bounded(&sh.load_q, phase, abort_flag)) failed = true;
      if (warp == 0) {
        tc::fence_after_sync();
        const uint32_t id = tc::idesc(tc::kBF16, 64, 64);
#pragma unroll 1
        for (int k = 0; k < 8; ++k)
          tc::mma_f16_elect(tb + kColX, tc::sdesc_at(dQ, 64, k), tc::sdesc_at(dK, 64, k), id, k > 0);
        tc::mma_commit_elect(&sh.scores);
      } else if (warp == 2) {
        tc::fence_after_sync();
        const uint32_t id = tc::idesc(tc::kBF16, 128, 64);
#pragma unroll 1
        for (int k = 0; k < (CORE ? 16 : 8); ++k)
          tc::mma_f16_ts_elect(tb + kColO1, tb + kColS + 8 * k, tc::sdesc_at(dQ, 64, k & 7), id, k > 0);
        tc::mma_commit_elect(&sh.outs);
      }
    }
    if (warp == kGateWarp) {
      const Two gl = G[kTc - 1];
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        const int t = lane + 32 * i;
        const Two a = G[t];
        if (MODE == kTWhole) sh.E[t] = p.scale * exp2_fast(a.hi + a.lo);
        sh.dk[t] = t < n ? exp2_fast((gl.hi - a.hi) + (gl.lo - a.lo)) : 0.f;
      }
    }
    // v: rows past the chunk's tokens are another sequence's (or stale): 0
    // there; non-finite elements are noted and replaced by 0
    if (MODE == kTWhole || n < kTc) {
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int u = tid + i * kTThreads, row = u >> 4, c16 = u & 15;
        uint4* at = reinterpret_cast<uint4*>(vt + (c16 >> 3) * 8192 + row * 128 + (((c16 & 7) ^ (row & 7)) << 4));
        uint4 x = *at;
        uint32_t* w = &x.x;
        uint32_t hit = 0;  // an exponent of all ones carries into the sign's place
#pragma unroll
        for (int e = 0; e < 4; ++e) hit |= (w[e] & 0x7f807f80u) + 0x00800080u;
        if (row >= n) {
          *at = make_uint4(0, 0, 0, 0);
        } else if (MODE == kTWhole && (hit & 0x80008000u) != 0) {
#pragma unroll
          for (int e = 0; e < 8; ++e)
            if (((w[e >> 1] >> (16 * (e & 1))) & 0x7f80u) == 0x7f80u) {
              atomicMin(&sh.bad[phase][8 * c16 + e], row);
              w[e >> 1] &= e & 1 ? 0x0000ffffu : 0xffff0000u;
            }
          *at = x;
          sh.any_bad[phase] = 1;
        }
      }
    }

    if (MODE == kTWhole) {
      if (!mbar_wait_bounded(&sh.scores, phase, abort_flag)) failed = true;
      tc::fence_after_sync();
      float x[16];
      tmem_ld_16x32(tq + kColX + 32 * hh, x);
      tc::tmem_wait_ld();
      const int ta = 16 * qd + (lane >> 2), s0 = 32 * hh + 2 * (lane & 3);  // rows ta and ta + 8
      const Two ga = G[ta], gb = G[ta + 8];
      unsigned char* pp = sm + kOffP + ta * 128 + 4 * (lane & 3);  // the rows are eight apart: the same swizzle
#pragma unroll
      for (int c = 0; c < 4; ++c) {
        const int sc = s0 + 8 * c;
        const Two u0 = G[sc], u1 = G[sc + 1];
        float2 y = make_float2(x[4 * c] * exp2_fast((ga.hi - u0.hi) + (ga.lo - u0.lo)),
                               x[4 * c + 1] * exp2_fast((ga.hi - u1.hi) + (ga.lo - u1.lo)));
        float2 z = make_float2(x[4 * c + 2] * exp2_fast((gb.hi - u0.hi) + (gb.lo - u0.lo)),
                               x[4 * c + 3] * exp2_fast((gb.hi - u1.hi) + (gb.lo - u1.lo)));
        y = mul2(y, p.scale);
        z = mul2(z, p.scale);
        if (sc > ta) y.x = 0.f;
        if (sc + 1 > ta) y.y = 0.f;
        if (sc > ta + 8) z.x = 0.f;
        if (sc + 1 > ta + 8) z.y = 0.f;
        unsigned char* at = pp + (((4 * hh + c) ^ (ta & 7)) << 4);
        *reinterpret_cast<uint32_t*>(at) = CORE ? split2(y) : pack2(y);
        *reinterpret_cast<uint32_t*>(at + 1024) = CORE ? split2(z) : pack2(z);
        if (CORE) {
          *reinterpret_cast<uint32_t*>(at + 8192) = pack2(y);
          *reinterpret_cast<uint32_t*>(at + 8192 + 1024) = pack2(z);
        }
      }
      fence_proxy_async_smem();
      tc::fence_before_sync();
      __syncthreads();  // #2: P and v are in shared memory, the scores are read
      if (warp == 4) {
        tc::fence_after_sync();
        const uint32_t id = tc::idesc(tc::kBF16, 128, 64) | kTransA;
#pragma unroll 1
        for (int k = 0; k < (CORE ? 8 : 4); ++k)
          tc::mma_f16_elect(tb + kColX, dV + ((k & 3) * 2048 >> 4), dP + (((k >> 2) * 8192 + (k & 3) * 32) >> 4), id,
                            k > 0);
        tc::mma_commit_elect(&sh.outs);
      }
    } else {
      if (n < kTc) fence_proxy_async_smem();
      __syncthreads();  // dk is in shared memory
    }

    // K' = e^(G_n - G_s) k in three parts, the first in place of K
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int u = tid + i * kTThreads, row = u >> 4, c16 = u & 15;
      const uint32_t off = (c16 >> 3) * 8192 + row * 128 + (((c16 & 7) ^ (row & 7)) << 4);
      uint4 x = *reinterpret_cast<const uint4*>(kt + off);
      if (row >= n) x = make_uint4(0, 0, 0, 0);  // another sequence's: may be a NaN
      const uint32_t* w = &x.x;
      const float d = sh.dk[row];
      uint4 part[3];
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        float2 a = mul2(unpack2(w[e]), d);
        (&part[0].x)[e] = cut2(a);
        (&part[1].x)[e] = cut2(a);
        (&part[2].x)[e] = __byte_perm(__float_as_uint(a.x), __float_as_uint(a.y), 0x7632);
      }
      *reinterpret_cast<uint4*>(kt + off) = part[0];
      *reinterpret_cast<uint4*>(sm + kOffMid + off) = part[1];
      *reinterpret_cast<uint4*>(sm + kOffLo + off) = part[2];
    }
    fence_proxy_async_smem();
    if (MODE == kTWhole) {  // for the next chunk, which writes them after #1
      if (tid < kTd) sh.bad[phase ^ 1][tid] = kTc;
      if (tid == 0) sh.any_bad[phase ^ 1] = 0;
    }
    if (MODE == kTWhole) {
      if (!mbar_wait_bounded(&sh.outs, phase, abort_flag)) failed = true;
      tc::fence_after_sync();
      if (tid == 0 && more) load_q(t0 + kTc);
      if (GATED && !mbar_wait_bounded(&sh.load_z, phase, abort_flag)) failed = true;
      // a lane holds value rows jj + 8 b + 16 a (a, b of 0, 1) and tokens
      // tt + 8 c, tt + 8 c + 1 (c of 0..3)
      const int jj = 32 * qd + (lane >> 2), tt = 32 * hh + 2 * (lane & 3);
      // o[2 c + b]: tokens tt + 8 c and the next, value row jj + 8 b + 16 a
      auto read_half = [&](int a, float2 (&o)[8]) {
        float x[16], y[16];
        tmem_ld_16x32(tq + ((uint32_t)(16 * a) << 16) + kColO1 + 32 * hh, x);
        tmem_ld_16x32(tq + ((uint32_t)(16 * a) << 16) + kColX + 32 * hh, y);
        tc::tmem_wait_ld();
#pragma unroll
        for (int c = 0; c < 4; ++c) {
          const float2 e = *reinterpret_cast<const float2*>(&sh.E[tt + 8 * c]);
#pragma unroll
          for (int b = 0; b < 2; ++b)
            o[2 * c + b] = fma2(make_float2(x[4 * c + 2 * b], x[4 * c + 2 * b + 1]), e,
                                make_float2(y[4 * c + 2 * b], y[4 * c + 2 * b + 1]));
        }
        if (sh.any_bad[phase])
#pragma unroll
          for (int i = 0; i < 8; ++i) {
            const int bad = sh.bad[phase][jj + 16 * a + 8 * (i & 1)], t = tt + 8 * (i >> 1);
            if (t >= bad) o[i].x = __int_as_float(0x7fc00000);
            if (t + 1 >= bad) o[i].y = __int_as_float(0x7fc00000);
          }
      };
      float2 inv[4];
      if (GATED) {
        float2 sq[4];
#pragma unroll
        for (int c = 0; c < 4; ++c) sq[c] = make_float2(0.f, 0.f);
#pragma unroll
        for (int a = 0; a < 2; ++a) {
          float2 o[8];
          read_half(a, o);
#pragma unroll
          for (int i = 0; i < 8; ++i) sq[i >> 1] = fma2(o[i], o[i], sq[i >> 1]);
        }
#pragma unroll
        for (int d = 4; d < 32; d <<= 1)
#pragma unroll
          for (int c = 0; c < 4; ++c) {
            sq[c].x += __shfl_xor_sync(0xffffffffu, sq[c].x, d);
            sq[c].y += __shfl_xor_sync(0xffffffffu, sq[c].y, d);
          }
        if (lane < 4)
#pragma unroll
          for (int c = 0; c < 4; ++c) *reinterpret_cast<float2*>(&sh.red[qd][tt + 8 * c]) = sq[c];
        asm volatile("bar.sync %0, 128;" ::"r"(1 + hh) : "memory");
#pragma unroll
        for (int c = 0; c < 4; ++c) {
          float2 r = make_float2(0.f, 0.f);
#pragma unroll
          for (int w = 0; w < 4; ++w) {
            const float2 x = *reinterpret_cast<const float2*>(&sh.red[w][tt + 8 * c]);
            r.x += x.x, r.y += x.y;
          }
          inv[c] = make_float2(rsqrtf(r.x * (1.f / kTd) + p.rms_eps), rsqrtf(r.y * (1.f / kTd) + p.rms_eps));
        }
      }
#pragma unroll
      for (int a = 0; a < 2; ++a) {
        float2 o[8];
        read_half(a, o);
        if (CORE)
#pragma unroll
          for (int i = 0; i < 8; ++i) {
            const int t = tt + 8 * (i >> 1);
            float* at = p.core_out + ((int64_t)(t0 + t) * p.Hv + h) * kTd + jj + 16 * a + 8 * (i & 1);
            if (t < n) at[0] = o[i].x;
            if (t + 1 < n) at[p.Hv * kTd] = o[i].y;
          }
        // blocks (rows jj block 0 and 1 of this half) x (token blocks 2 d, 2 d + 1)
#pragma unroll
        for (int d = 0; d < 2; ++d) {
          const int t = 32 * hh + 16 * d + 8 * (lane >> 4) + (lane & 7), c8 = 4 * qd + 2 * a + ((lane >> 3) & 1);
          const uint32_t at = smem_u32(sm + kOffO) + (c8 >> 3) * 8192 + t * 128 + (((c8 & 7) ^ (t & 7)) << 4);
          uint32_t r[4];
          if (GATED) {
            ldmatrix_t4(at, r);
            const float w0 = sh.w[jj + 16 * a], w1 = sh.w[jj + 16 * a + 8];
#pragma unroll
            for (int m = 0; m < 4; ++m) {
              const float2 z = unpack2(r[m]);
              const float2 e = mul2(z, -kLog2e);
              const float2 den = make_float2(1.f + exp2_fast(e.x), 1.f + exp2_fast(e.y));
              const float2 silu = make_float2(__fdividef(z.x, den.x), __fdividef(z.y, den.y));
              const float2 g = fma2(silu, mul2(inv[2 * d + (m >> 1)], m & 1 ? w1 : w0), make_float2(-0.f, -0.f));
              o[4 * d + m] = fma2(o[4 * d + m], g, make_float2(-0.f, -0.f));
            }
          }
#pragma unroll
          for (int m = 0; m < 4; ++m) r[m] = pack2(o[4 * d + m]);
          stmatrix_t4(at, r);
        }
      }
      fence_proxy_async_smem();
    }
    tc::fence_before_sync();
    __syncthreads();  // #3: K' is in shared memory, the outputs are staged and their TMEM columns read
    if (warp == kDeltaWarp) {
      tc::fence_after_sync();
      const uint32_t id = tc::idesc(tc::kBF16, 128, 128) | kTransA | kTransB;
      const uint64_t dK0 = sdesc_mn128(smem_u32(kt));
#pragma unroll 1
      for (int k = 0; k < 12; ++k)
        tc::mma_f16_elect(tb + kColX, dV + ((k & 3) * 2048 >> 4),
                          (k < 4 ? dK0 : dMid + (k < 8 ? 0 : kTile16 >> 4)) + ((k & 3) * 2048 >> 4), id, k > 0);
      tc::mma_commit_elect(&sh.delta);
    } else if (warp == kGateWarp) {
      if (more) {
        // one decay for all tokens: full chunks share their sums, in both buffers after the second
        if (p.g_stride != 0 || t0 == s.begin || tokens(t0 + kTc) < kTc) put_sums(sh.G[phase ^ 1]);
        if (MODE == kTLocal) total = add2(total, gn);
        fetch_g(t0 + 2 * kTc);
      }
    } else if (MODE == kTWhole && (!CORE || p.out != nullptr)) {
      if (n == kTc) {
        if (warp == kStoreWarp && lane == 0) {
          for (int b = 0; b < 2; ++b) tc::tma_store_2d(&tm_o, h * kTd + 64 * b, t0, sm + kOffO + 8192 * b);
          bulk_commit();
          bulk_wait_read_all();
        }
      } else if (warp != 7) {
        // a last, shorter chunk: its rows alone, by the warps 0, 2, 3, 4 and 5
        const int first = warp == 0 ? 0 : warp - 1;
        for (int u = first * 32 + lane; u < 16 * n; u += 5 * 32) {
          const int t = u >> 4, c8 = u & 15;
          *reinterpret_cast<uint4*>(static_cast<__nv_bfloat16*>(p.out) + ((int64_t)(t0 + t) * p.Hv + h) * kTd + 8 * c8) =
              *reinterpret_cast<const uint4*>(sm + kOffO + (c8 >> 3) * 8192 + t * 128 + (((c8 & 7) ^ (t & 7)) << 4));
        }
      }
    }
    if (GATED && more && warp == kStoreWarp && lane == 0) load_z(t0 + kTc);
    const Decay a = decay_factor((G[kTc - 1].hi + G[kTc - 1].lo) * kLn2);
    if (!mbar_wait_bounded(&sh.delta, phase, abort_flag)) failed = true;
    tc::fence_after_sync();
    if (tid == 0 && (MODE == kTLocal ? t0 + 2 * kTc < s.end : more)) load_kv(t0 + (MODE == kTLocal ? 2 : 1) * kTc, stage);
    {
      const float2 f = make_float2(a.factor, a.factor), keep = make_float2(a.keep, a.keep);
      const bool spoilt = MODE == kTWhole && sh.any_bad[phase] && sh.bad[phase][j] < kTc;
#pragma unroll
      for (int c = 0; c < 2; ++c) {
        float d[32];
        tc::tmem_ld16(tq + kColX + 64 * hh + 32 * c, *reinterpret_cast<float(*)[16]>(d));
        tc::tmem_ld16(tq + kColX + 64 * hh + 32 * c + 16, *reinterpret_cast<float(*)[16]>(d + 16));
        tc::tmem_wait_ld();
        if (a.keep != 0.f) {
#pragma unroll
          for (int e = 0; e < 16; ++e)
            S[16 * c + e] = fma2(f, S[16 * c + e], fma2(keep, S[16 * c + e], make_float2(d[2 * e], d[2 * e + 1])));
        } else {
#pragma unroll
          for (int e = 0; e < 16; ++e) S[16 * c + e] = fma2(f, S[16 * c + e], make_float2(d[2 * e], d[2 * e + 1]));
        }
        if (spoilt)
#pragma unroll
          for (int e = 0; e < 16; ++e) S[16 * c + e] = make_float2(__int_as_float(0x7fc00000), __int_as_float(0x7fc00000));
        if (MODE == kTWhole && more) put_state(c);
      }
      if (MODE == kTWhole && more) tc::tmem_wait_st();
    }
    tc::fence_before_sync();
    // #1 of the next chunk: everything of this one is read
    if (__syncthreads_or(failed)) break;
  }

  if (!failed && !*abort_flag) {
    if (MODE == kTLocal || s.index + 1 == s.parts) {
      float* to = MODE == kTLocal ? sg.states + (int64_t)blockIdx.x * (kTd * kTd) : gS;
#pragma unroll
      for (int c = 0; c < 8; ++c)
        store8(to + at0 + 8 * c, make_float4(S[4 * c].x, S[4 * c].y, S[4 * c + 1].x, S[4 * c + 1].y),
               make_float4(S[4 * c + 2].x, S[4 * c + 2].y, S[4 * c + 3].x, S[4 * c + 3].y));
    }
    if (MODE == kTLocal && warp == 1 && lane == 0) sg.decays[blockIdx.x] = exp2f(total.hi + total.lo);
  }
  // no load may still be in flight when the CTA ends: after a wait that gave
  // up the next chunk's may be
  if (tid == 0) {
    if (MODE == kTLocal) {  // load i goes to stage i % 2
      mbar_wait(&sh.load_kv[0], ((kv_loads + 1) / 2 - 1) & 1);
      if (kv_loads > 1) mbar_wait(&sh.load_kv[1], (kv_loads / 2 - 1) & 1);
    } else {
      mbar_wait(&sh.load_kv[0], (kv_loads - 1) & 1);
    }
    if (MODE == kTWhole) mbar_wait(&sh.load_q, (q_loads - 1) & 1);
  }
  if (MODE == kTWhole && warp == kStoreWarp && lane == 0) {
    if (GATED) mbar_wait(&sh.load_z, (z_loads - 1) & 1);
    bulk_wait_all();
  }
  tc::fence_before_sync();
  __syncthreads();
  if (warp == 0) {
    tc::fence_after_sync();
    tc::tmem_dealloc(tb, kCols);
  }
}

}  // namespace

bool decay_tc_fits(int32_t dtype, int32_t D) { return dtype == GDN_BF16 && D == kTd; }

bool decay_tc_supported(const DecayArgs& p) {
  // states are read and written in 32-byte accesses
  return reinterpret_cast<uintptr_t>(p.state) % 32 == 0 && tc::encode_fn() != nullptr;
}

cudaError_t launch_decay_tc(const DecayArgs& p, const DecaySegments& sg, cudaStream_t stream) {
  const CUtensorMapDataType bf = CU_TENSOR_MAP_DATA_TYPE_BFLOAT16;
  CUtensorMap mq, mk, mv, mz{}, mo{};
  bool mz_ok, mo_ok;
  if (!tc::make_map_2d(&mq, p.q, p.T, (int64_t)p.Hk * kTd, p.q_stride, 2, bf, 64, kTc, CU_TENSOR_MAP_SWIZZLE_128B) ||
      !tc::make_map_2d(&mk, p.k, p.T, (int64_t)p.Hk * kTd, p.k_stride, 2, bf, 64, kTc, CU_TENSOR_MAP_SWIZZLE_128B) ||
      !tc::make_map_2d(&mv, p.v, p.T, (int64_t)p.Hv * kTd, p.v_stride, 2, bf, 64, kTc, CU_TENSOR_MAP_SWIZZLE_128B))
    return cudaErrorInvalidValue;
  // z and out: the maps of those that are not there are never used
  mz_ok = p.z == nullptr || tc::make_map_2d(&mz, p.z, p.T, (int64_t)p.Hv * kTd, p.z_stride, 2, bf, 64, kTc,
                                            CU_TENSOR_MAP_SWIZZLE_128B);
  mo_ok = p.out == nullptr || tc::make_map_2d(&mo, p.out, p.T, (int64_t)p.Hv * kTd, (int64_t)p.Hv * kTd, 2, bf, 64, kTc,
                                              CU_TENSOR_MAP_SWIZZLE_128B);
  if (!mz_ok || !mo_ok) return cudaErrorInvalidValue;
  const unsigned grid = (unsigned)(sg.slots * p.Hv);
  const auto run = [&](auto* kernel, bool core) {
    const int smem = (int)tc_smem(core) + 1024;
    const cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
    if (e != cudaSuccess) return e;
    kernel<<<grid, kTThreads, smem, stream>>>(p, sg, mq, mk, mv, mz, mo);
    return cudaGetLastError();
  };
  if (sg.states != nullptr) {
    const cudaError_t e = run(decay_tc_kernel<kTLocal, false, false>, false);
    if (e != cudaSuccess) return e;
  }
  if (p.core_out != nullptr)
    return p.z != nullptr ? run(decay_tc_kernel<kTWhole, true, true>, true) : run(decay_tc_kernel<kTWhole, true, false>, true);
  return p.z != nullptr ? run(decay_tc_kernel<kTWhole, false, true>, false)
                        : run(decay_tc_kernel<kTWhole, false, false>, false);
}

}  // namespace gdn

GDN_DEFINE_ERROR_READER(decay_tc)
