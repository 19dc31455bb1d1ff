// Shared device code of linear attention with a decay for each head:
//   S_t[j][i] = exp(g_t) S_{t-1}[j][i] + v_t[j] k_t[i],  o_t[j] = scale sum_i S_t[j][i] q_t[i]
// over the library's fp32 states S[h][j][i] (value row j, key column i).
#pragma once

#include "gdn_common.cuh"
#include "gdn_internal.h"

namespace gdn {

// exp(g) is 0 in fp32 from about -104 on, so a log decay below this bound
// acts exactly as the bound does; bounding it keeps sums of log decays finite
// (g = -inf is a reset of the state). A NaN stays one.
constexpr float kDecayFloor = -128.f;
__device__ __forceinline__ float decay_log(float g) { return g < kDecayFloor ? kDecayFloor : g; }

// s <- exp(g) s + d v on a lane's groups. Near 1 the factor's own rounding
// would add up over a long memory (1000 tokens of it at g = -0.001 are 3e-5),
// so from one half up s + expm1(g) s is taken instead, whose error is a
// rounding of the result alone: keep is 1 and factor expm1(g) there, else 0
// and exp(g), two FMAs an element either way.
struct Decay {
  float keep, factor;
};
__device__ __forceinline__ Decay decay_factor(float g) {
  return g > -0.69f ? Decay{1.f, expm1f(g)} : Decay{0.f, expf(g)};
}
template <int NV4>
__device__ __forceinline__ void decay_update_near(float4 (&s)[NV4], const float4 (&v)[NV4], float factor, float d) {
  const float2 al = make_float2(factor, factor), dd = make_float2(d, d);
#pragma unroll
  for (int m = 0; m < NV4; ++m) {
    const float2 s0 = make_float2(s[m].x, s[m].y), s1 = make_float2(s[m].z, s[m].w);
    const float2 lo = fma2(dd, make_float2(v[m].x, v[m].y), fma2(al, s0, s0));
    const float2 hi = fma2(dd, make_float2(v[m].z, v[m].w), fma2(al, s1, s1));
    s[m] = make_float4(lo.x, lo.y, hi.x, hi.y);
  }
}
template <int NV4>
__device__ __forceinline__ void decay_update(float4 (&s)[NV4], const float4 (&v)[NV4], Decay a, float d) {
  if (a.keep == 0.f) row_update<NV4>(s, v, a.factor, d);
  else decay_update_near<NV4>(s, v, a.factor, d);
}

// How the D x D state of a head lies over the threads of a CTA: LPR lanes
// share a row, each with NV4 groups of four columns (group m of lane sub at
// column 4 sub + 4 LPR m, so that the lanes of a row read 64 or 128
// contiguous bytes at a time); a lane has RPL rows, RPW apart: fewer (FEW)
// where few CTAs run and a token's latency counts, not what it issues.
template <int D, bool FEW = false>
struct DecayGeom {
  static constexpr int LPR = D == 32 ? 4 : (D == 64 ? 4 : 8);
  static constexpr int NV4 = D / (4 * LPR);
  static constexpr int RPW = 32 / LPR;
  static constexpr int RPL = FEW ? (D == 128 || D == 96 ? 2 : 1) : (D == 32 ? 2 : (D == 96 ? 3 : 4));
  static constexpr int WROWS = RPW * RPL;  // rows a warp owns
  static constexpr int WARPS = D / WROWS;
  static constexpr int THREADS = 32 * WARPS;
  static_assert(WARPS * WROWS == D, "the warps' rows cover the state");
};

// four consecutive elements as fp32 (16-byte, or 8-byte aligned for 16-bit types)
template <typename T>
__device__ __forceinline__ float4 load4(const T* p);
template <>
__device__ __forceinline__ float4 load4<float>(const float* p) {
  return *reinterpret_cast<const float4*>(p);
}
template <>
__device__ __forceinline__ float4 load4<__half>(const __half* p) {
  const uint2 u = *reinterpret_cast<const uint2*>(p);
  const float2 a = __half22float2(*reinterpret_cast<const __half2*>(&u.x));
  const float2 b = __half22float2(*reinterpret_cast<const __half2*>(&u.y));
  return make_float4(a.x, a.y, b.x, b.y);
}
template <>
__device__ __forceinline__ float4 load4<__nv_bfloat16>(const __nv_bfloat16* p) {
  const uint2 u = *reinterpret_cast<const uint2*>(p);
  return make_float4(__uint_as_float(u.x << 16), __uint_as_float(u.x & 0xffff0000u),
                     __uint_as_float(u.y << 16), __uint_as_float(u.y & 0xffff0000u));
}

// Outputs of one (token, V head): o[D] in shared memory (already scaled);
// one warp, D/32 consecutive elements a lane. core_out, out and z point at
// the row; z == nullptr: out is o rounded once.
template <typename T, int D>
__device__ __forceinline__ void decay_write_row(const float* o, float* core_out, const T* z,
                                                const float* norm_w, T* out, float rms_eps, int lane) {
  constexpr int PER = D / 32;
  float ov[PER];
#pragma unroll
  for (int e = 0; e < PER; ++e) ov[e] = o[lane * PER + e];
  if (core_out != nullptr) {
#pragma unroll
    for (int e = 0; e < PER; ++e) core_out[lane * PER + e] = ov[e];
  }
  if (out == nullptr) return;
  if (z != nullptr) {
    float ss = 0.f;
#pragma unroll
    for (int e = 0; e < PER; ++e) ss += ov[e] * ov[e];
    ss = group_sum<32>(ss);
    const float inv = 1.f / sqrtf(ss / (float)D + rms_eps);
#pragma unroll
    for (int e = 0; e < PER; ++e)
      ov[e] = ov[e] * inv * norm_w[lane * PER + e] * silu_f(to_f32(z[lane * PER + e]));
  }
#pragma unroll
  for (int e = 0; e < PER; ++e) out[lane * PER + e] = from_f32<T>(ov[e]);
}

// eight consecutive floats as one 32-byte access
__device__ __forceinline__ void load8(const float* p, float4& a, float4& b) {
  asm volatile("ld.global.v8.f32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8];"
               : "=f"(a.x), "=f"(a.y), "=f"(a.z), "=f"(a.w), "=f"(b.x), "=f"(b.y), "=f"(b.z), "=f"(b.w)
               : "l"(p));
}
__device__ __forceinline__ void store8(float* p, float4 a, float4 b) {
  asm volatile("st.global.v8.f32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(p), "f"(a.x), "f"(a.y), "f"(a.z),
               "f"(a.w), "f"(b.x), "f"(b.y), "f"(b.z), "f"(b.w)
               : "memory");
}

// ------------------------------------------------------------- segments
// Sequences of more than sg.whole tokens are cut into segments of sg.len, the
// others are one segment each. Segment i of sequence n has slot
//   floor(cu[n] / len) + n + i,
// which is increasing and never reaches the next sequence's first slot
// (ceil((b - a) / len) <= floor(b / len) - floor(a / len) + 1), so
// floor(T / len) + N slots hold every segment, the host need not know the
// lengths, and a slot finds its sequence by a search over cu_seqlens.
// In the workspace only the sequences that are cut have slots. Each of them
// is longer than whole, so they can be told apart by floor(cu[n] / whole), too:
// where that is fewer than N, segment i has workspace slot
//   floor(cu[n] / len) + floor(cu[n] / whole) + i
// (the next cut sequence begins more than whole later), below
// floor(T / len) + floor(T / whole), whatever cu holds.

__device__ __forceinline__ int seq_bound(const DecayArgs& p, int n) {
  const int c = p.cu_seqlens[n];
  return c < 0 ? 0 : (c > p.T ? p.T : c);
}
__device__ __forceinline__ int seq_end(const DecayArgs& p, int n, int begin) {
  const int c = seq_bound(p, n + 1);
  return c < begin ? begin : c;
}

struct DecaySegment {
  int seq;
  int index, parts;    // which of the sequence's segments, and how many it has
  int kept;            // of its first segment in the workspace, if it has several
  int begin, end;      // tokens
};

// The segment of a slot; false where the slot is spare or its sequence is
// empty. Every lane of a warp calls it: the warp probes 32 sequences at a
// time, so that up to 32 sequences take one load and up to 1024 two.
__device__ __forceinline__ bool find_segment(const DecayArgs& p, const DecaySegments& sg, int slot, int lane,
                                             DecaySegment* out) {
  int lo = 0, count = p.N;  // the last sequence in [lo, lo + count) whose first slot is <= slot
  while (count > 1) {
    const int step = (count + 31) / 32;
    const int n = lo + lane * step;
    const bool le = lane * step < count && seq_bound(p, n) / sg.len + n <= slot;
    const unsigned hits = __ballot_sync(0xffffffffu, le);
    const int at = hits == 0 ? 0 : 31 - __clz(hits);
    lo += at * step;
    count = count - at * step < step ? count - at * step : step;
  }
  const int begin = seq_bound(p, lo), end = seq_end(p, lo, begin);
  const int length = end - begin;
  out->kept = begin / sg.len + (sg.whole > p.T / p.N ? begin / sg.whole : lo);
  out->parts = length <= sg.whole ? (length > 0 ? 1 : 0) : 1 + (length - 1) / sg.len;
  const int i = slot - (begin / sg.len + lo);
  if (i < 0 || i >= out->parts) return false;
  out->seq = lo;
  out->index = i;
  out->begin = begin + i * sg.len;
  out->end = i + 1 == out->parts ? end : out->begin + sg.len;
  return true;
}

// The first pass over a sequence of several segments leaves in its slot m of
// the workspace what segment m adds to the state (segment 0: the state after it)
// and in decays[m] what it multiplies the state by. The last segment is not
// in that pass; its slot keeps a copy of the state before the call, which
// the call overwrites. These read and write four elements at `at` of V head
// h's state.
struct DecaySlots {
  const float* base;  // slot of segment 0, V head h
  int64_t step;       // floats between slots
  const float* decay;
  int32_t dstep;
  __device__ __forceinline__ DecaySlots(const DecayArgs& p, const DecaySegments& sg, const DecaySegment& s, int h,
                                        int dd) {
    base = sg.states + ((int64_t)s.kept * p.Hv + h) * dd;
    step = (int64_t)p.Hv * dd;
    decay = sg.decays + ((int64_t)s.kept * p.Hv + h);
    dstep = p.Hv;
  }
  // n times eight elements from `at`, for a thread that holds part of a row:
  // whole 32-byte sectors, the loads of a segment in flight together
  template <int N>
  __device__ __forceinline__ void start8(int i, int parts, int at, float4 (&s)[2 * N]) const {
    const float* first = base + (i == 0 ? (parts - 1) * step : 0) + at;
#pragma unroll
    for (int c = 0; c < N; ++c) load8(first + 8 * c, s[2 * c], s[2 * c + 1]);
    for (int m = 1; m < i; ++m) {
      const float a = decay[m * dstep];
      float4 x[2 * N];
#pragma unroll
      for (int c = 0; c < N; ++c) load8(base + m * step + at + 8 * c, x[2 * c], x[2 * c + 1]);
#pragma unroll
      for (int c = 0; c < 2 * N; ++c)
        s[c] = make_float4(fmaf(a, s[c].x, x[c].x), fmaf(a, s[c].y, x[c].y), fmaf(a, s[c].z, x[c].z),
                           fmaf(a, s[c].w, x[c].w));
    }
  }
  // four elements at each of N places at + c * stride of the state at the start
  // of segment i, the loads of a segment in flight together
  template <int N>
  __device__ __forceinline__ void start4(int i, int parts, int at, int stride, float4 (&s)[N]) const {
    const float* first = base + (i == 0 ? (parts - 1) * step : 0) + at;
#pragma unroll
    for (int c = 0; c < N; ++c) s[c] = *reinterpret_cast<const float4*>(first + c * stride);
    for (int m = 1; m < i; ++m) {
      const float a = decay[m * dstep];
      float4 x[N];
#pragma unroll
      for (int c = 0; c < N; ++c) x[c] = *reinterpret_cast<const float4*>(base + m * step + at + c * stride);
#pragma unroll
      for (int c = 0; c < N; ++c)
        s[c] = make_float4(fmaf(a, s[c].x, x[c].x), fmaf(a, s[c].y, x[c].y), fmaf(a, s[c].z, x[c].z),
                           fmaf(a, s[c].w, x[c].w));
    }
  }
};

}  // namespace gdn
