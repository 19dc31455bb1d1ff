// Rotary positions of queries and keys, with the keys and values going to the
// rows of a cache where one is given:
//   y1 = a (x1 cos t - x2 sin t),  y2 = a (x2 cos t + x1 sin t),  t = position x frequency
// for each pair (x1, x2) of a head's first rotary_dim elements; the rest of
// the head is copied.
//
// An angle is a fraction of a turn, held as a 64-bit integer (2^64 one turn):
// position times the pair's step modulo 2^64 is that fraction exactly, however
// far the position is, where a product in fp32 would have lost it (2^-24 of
// 10^6 turns is a sixteenth of one). The step is the frequency rounded to 2^-64
// of a turn (rope_steps.cu), the fraction at 2^-24 of itself, then sincospif.
//
// A CTA takes one token or a few and puts the sines and cosines of their pairs
// into shared memory. A thread has the same elements of every so-many-th head
// of q, k and v of one token: 16 bytes (two times 16 where the pairs are
// halves; single elements where a half ends within 16 bytes), and so keeps
// their sines and cosines in registers. 8192 tokens of 64 + 8 heads of 128:
//   bf16, halves, the whole head      56 us, 5.35 TB/s: bound by memory
//   bf16, halves, 64 of 128 turn      76 us, 4.0 TB/s
//   bf16, neighbours, all or a part   75 us, 4.0 TB/s
//   bf16, halves of 18                178 us, 1.7 TB/s: 2 bytes an access
//   fp32, halves of 18                190 us, 3.2 TB/s: 4 bytes an access
// (16-bit halves of 16 bytes spill 8 bytes under the bound of four CTAs an SM.)
#include <type_traits>

#include "gdn_common.cuh"
#include "gdn_internal.h"

namespace gdn {
namespace {

constexpr int kRThreads = 256;  // at most
constexpr int kRMaxTokens = 16;
constexpr int kRMaxPairs = 64;

template <typename T>
struct alignas(16) Vec {
  static constexpr int N = 16 / (int)sizeof(T);
  T e[N];
};

template <typename T>
struct Single {
  T e[1];
};

// two neighbouring elements as fp32, and back
template <typename T>
__device__ __forceinline__ float2 get2(const T* p) {
  return make_float2(to_f32(p[0]), to_f32(p[1]));
}
template <>
__device__ __forceinline__ float2 get2<__nv_bfloat16>(const __nv_bfloat16* p) {
  const uint32_t u = *reinterpret_cast<const uint32_t*>(p);
  return make_float2(__uint_as_float(u << 16), __uint_as_float(u & 0xffff0000u));
}
template <>
__device__ __forceinline__ float2 get2<__half>(const __half* p) {
  return __half22float2(*reinterpret_cast<const __half2*>(p));
}
template <typename T>
__device__ __forceinline__ void put2(T* p, float2 x) {
  p[0] = from_f32<T>(x.x), p[1] = from_f32<T>(x.y);
}
template <>
__device__ __forceinline__ void put2<__nv_bfloat16>(__nv_bfloat16* p, float2 x) {
  *reinterpret_cast<__nv_bfloat162*>(p) = __float22bfloat162_rn(x);
}
template <>
__device__ __forceinline__ void put2<__half>(__half* p, float2 x) {
  *reinterpret_cast<__half2*>(p) = __float22half2_rn(x);
}

// What a head's units are: those that rotate, then those that copy.
struct RopeShape {
  int tokens;  // a CTA
  int heads;   // that lie side by side over the threads of a token
  int turn, copy;
};

template <typename T, bool HALF, bool VECTOR>
__global__ void __launch_bounds__(kRThreads, 4) rope_kernel(const RopeArgs p, const RopeShape sh) {
  constexpr int V = VECTOR ? Vec<T>::N : 1, PAIRS = HALF ? V : V / 2;
  using E = typename std::conditional<VECTOR, Vec<T>, Single<T>>::type;
  __shared__ float2 cs[kRMaxTokens][kRMaxPairs];
  const int tid = threadIdx.x, pairs = p.table.rotary_dim / 2;
  const int64_t t0 = (int64_t)blockIdx.x * sh.tokens;
  const int n = p.T - t0 < sh.tokens ? (int)(p.T - t0) : sh.tokens;
  const int per = sh.turn + sh.copy, w = tid % per, th = tid / per;
  const int t = th / sh.heads, h0 = th % sh.heads + blockIdx.y * sh.heads, step = gridDim.y * sh.heads;
  const int hq = p.q != nullptr ? p.Hq : 0, hk = p.k != nullptr ? p.Hk : 0, hv = p.v != nullptr ? p.Hk : 0;
  const int heads = t < n ? hq + hk + hv : 0;
  const bool two = HALF && w < sh.turn;  // a at `at`, b half of the pairs behind it
  const int at = !HALF || two ? w * V : 2 * pairs + (w - sh.turn) * V;
  const int64_t token = t0 + t;
  int64_t row = token;  // of k_out and v_out; a padded token's key and value go nowhere
  if (p.cache_rows != nullptr && heads > 0) {
    row = p.cache_rows[token];
    if (row >= p.num_rows) {
      record_device_error(GDN_ERR_EXTENT);
      row = -1;
    }
  }
  const T* xq = static_cast<const T*>(p.q) + token * p.q_stride + at;
  const T* xk = static_cast<const T*>(p.k) + token * p.k_stride + at;
  const T* xv = static_cast<const T*>(p.v) + token * p.v_stride + at;
  T* yq = static_cast<T*>(p.q_out) + token * p.q_out_stride + at;
  T* yk = static_cast<T*>(p.k_out) + row * p.k_out_stride + at;
  T* yv = static_cast<T*>(p.v_out) + row * p.v_out_stride + at;
  const auto load = [&](int h, E& a, E& b) {
    const T* x = h < hq ? xq + h * p.D : h < hq + hk ? xk + (h - hq) * p.D : xv + (h - hq - hk) * p.D;
    a = *reinterpret_cast<const E*>(x);
    if (two) b = *reinterpret_cast<const E*>(x + pairs);
  };
  E a{}, b{};
  if (h0 < heads) load(h0, a, b);
  for (int i = tid; i < n * pairs; i += blockDim.x) {
    const int tt = i / pairs, pair = i % pairs;
    const uint64_t turn = (uint64_t)(int64_t)p.positions[t0 + tt] * p.table.step[pair];
    float s, c;
    sincospif(__ll2float_rn((long long)turn) * 1.0842021724855044e-19f, &s, &c);  // 2^-63: half turns
    cs[tt][pair] = make_float2(c * p.table.amplitude, (p.inverse ? -s : s) * p.table.amplitude);
  }
  __syncthreads();
  float c[PAIRS], d[PAIRS];              // cosines and sines
  const int first = HALF ? at : at / 2;  // of this thread's pairs
#pragma unroll
  for (int e = 0; e < PAIRS; ++e) {
    const bool pair = (!HALF || two) && first + e < pairs;
    const float2 f = pair ? cs[t < n ? t : 0][first + e] : make_float2(1.f, 0.f);
    c[e] = f.x, d[e] = f.y;
  }
  for (int h = h0; h < heads; h += step) {
    E na{}, nb{};
    if (h + step < heads) load(h + step, na, nb);
    if (h < hq + hk) {
      if (HALF && two) {
        if constexpr (PAIRS == 1) {
          const float x1 = to_f32(a.e[0]), x2 = to_f32(b.e[0]);
          a.e[0] = from_f32<T>(fmaf(x1, c[0], -(x2 * d[0])));
          b.e[0] = from_f32<T>(fmaf(x2, c[0], x1 * d[0]));
        } else {
#pragma unroll
          for (int e = 0; e < PAIRS; e += 2) {
            const float2 x1 = get2<T>(a.e + e), x2 = get2<T>(b.e + e), zero = make_float2(-0.f, -0.f);
            const float2 cc = make_float2(c[e], c[e + 1]), dd = make_float2(d[e], d[e + 1]);
            put2<T>(a.e + e, fma2(x1, cc, fma2(x2, make_float2(-dd.x, -dd.y), zero)));
            put2<T>(b.e + e, fma2(x2, cc, fma2(x1, dd, zero)));
          }
        }
      } else if (!HALF) {
#pragma unroll
        for (int e = 0; e < PAIRS; ++e)
          if (first + e < pairs) {
            const float2 x = get2<T>(a.e + 2 * e);
            put2<T>(a.e + 2 * e, make_float2(fmaf(x.x, c[e], -(x.y * d[e])), fmaf(x.y, c[e], x.x * d[e])));
          }
      }
    }
    if (h < hq || row >= 0) {
      T* y = h < hq ? yq + h * p.D : h < hq + hk ? yk + (h - hq) * p.D : yv + (h - hq - hk) * p.D;
      *reinterpret_cast<E*>(y) = a;
      if (two) *reinterpret_cast<E*>(y + pairs) = b;
    }
    a = na;
    b = nb;
  }
}

template <typename T>
cudaError_t run(const RopeArgs& p, cudaStream_t stream) {
  constexpr int V = Vec<T>::N;
  const int r = p.table.rotary_dim;
  const bool half = p.table.layout == GDN_ROPE_HALF, vector = !half || r / 2 % V == 0;
  RopeShape sh{};
  if (!half) {
    sh.turn = p.D / V;
  } else {
    sh.turn = r / 2 / (vector ? V : 1);
    sh.copy = (p.D - r) / (vector ? V : 1);
  }
  const int heads = (p.q ? p.Hq : 0) + (p.k ? p.Hk : 0) + (p.v ? p.Hk : 0);
  // a token: as many heads side by side as fit, in rounds of the same number
  const int per = sh.turn + sh.copy, fit = kRThreads / per;
  const int rounds = (heads + fit - 1) / fit;
  sh.heads = (heads + rounds - 1) / rounds;
  // few tokens: the rounds of one as CTAs of their own
  int parts = 1;
  while (parts < rounds && p.T * parts < 152) ++parts;
  // few heads: several tokens a CTA, but CTAs for all SMs first
  int64_t tokens = kRThreads / (per * sh.heads);
  tokens = tokens > kRMaxTokens ? kRMaxTokens : tokens;
  while (tokens > 1 && (p.T + tokens - 1) / tokens < 304) tokens /= 2;
  sh.tokens = (int)tokens;
  const unsigned threads = (unsigned)(per * sh.heads * sh.tokens);
  const dim3 grid((unsigned)((p.T + tokens - 1) / tokens), (unsigned)parts);
  if (!half) rope_kernel<T, false, true><<<grid, threads, 0, stream>>>(p, sh);
  else if (vector) rope_kernel<T, true, true><<<grid, threads, 0, stream>>>(p, sh);
  else rope_kernel<T, true, false><<<grid, threads, 0, stream>>>(p, sh);
  return cudaGetLastError();
}

}  // namespace

cudaError_t launch_rope(const RopeArgs& p, int32_t dtype, cudaStream_t stream) {
  switch (dtype) {
    case GDN_F16: return run<__half>(p, stream);
    case GDN_BF16: return run<__nv_bfloat16>(p, stream);
    default: return run<float>(p, stream);
  }
}

}  // namespace gdn

GDN_DEFINE_ERROR_READER(rope)
