// Rotary positions of queries and keys, with the keys and values going to the
// rows of a cache where one is given:
//   y1 = a (x1 cos t - x2 sin t),  y2 = a (x2 cos t + x1 sin t),  t = position x frequency
// for each pair (x1, x2) of a head's first rotary_dim elements; the rest of
// the head is copied.
//
// An angle is a fraction of a turn, held as a 64-bit integer (2^64 one turn):
// position times the pair's step modulo 2^64 is that fraction exactly, however
// far the position is, where a product in fp32 would have lost it (2^-24 of
// 10^6 turns is a sixteenth of one). The step is rounded at 2^-64 of a turn,
// the fraction at 2^-24 of itself, then sincospif.
//
// A CTA takes one token or a few, puts the sines and cosines of their pairs
// into shared memory and goes over all heads of q, k and v with 16-byte
// accesses (single elements where a half of the pairs ends within 16 bytes).
// Bound by memory.
#include "gdn_common.cuh"
#include "gdn_internal.h"

namespace gdn {
namespace {

constexpr int kRThreads = 256;
constexpr int kRMaxTokens = 16;
constexpr int kRMaxPairs = 64;

template <typename T>
struct alignas(16) Vec {
  static constexpr int N = 16 / (int)sizeof(T);
  T e[N];
};

// What a head's units are: those that rotate, then those that copy. VECTOR
// units are 16 bytes (two times 16 where the pairs are halves), else one pair
// or one element.
struct RopeShape {
  int tokens;  // a CTA
  int turn, copy;
};

template <typename T, bool HALF, bool VECTOR>
__global__ void __launch_bounds__(kRThreads) rope_kernel(const RopeArgs p, const RopeShape sh) {
  constexpr int V = Vec<T>::N;
  __shared__ float2 cs[kRMaxTokens][kRMaxPairs];
  const int tid = threadIdx.x;
  const int pairs = p.table.rotary_dim / 2;
  const int64_t t0 = (int64_t)blockIdx.x * sh.tokens;
  const int n = p.T - t0 < sh.tokens ? (int)(p.T - t0) : sh.tokens;
  for (int u = tid; u < n * pairs; u += kRThreads) {
    const int t = u / pairs, i = u % pairs;
    const uint64_t turn = (uint64_t)(int64_t)p.positions[t0 + t] * p.table.step[i];
    float s, c;
    sincospif(__ll2float_rn((long long)turn) * 1.0842021724855044e-19f, &s, &c);  // 2^-63: half turns
    cs[t][i] = make_float2(c * p.table.amplitude, (p.inverse ? -s : s) * p.table.amplitude);
  }
  __syncthreads();
  const int hq = p.q != nullptr ? p.Hq : 0, hk = p.k != nullptr ? p.Hk : 0, hv = p.v != nullptr ? p.Hk : 0;
  const int per = sh.turn + sh.copy, heads = hq + hk + hv;
  const int units = n * heads * per;
  for (int u = blockIdx.y * kRThreads + tid; u < units; u += gridDim.y * kRThreads) {
    const int w = u % per, th = u / per;
    int h = th % heads;
    const int t = th / heads;
    const int64_t token = t0 + t;
    const T* x;
    T* y;
    bool value = false;
    if (h < hq) {
      x = static_cast<const T*>(p.q) + token * p.q_stride;
      y = static_cast<T*>(p.q_out) + token * p.q_out_stride;
    } else {
      h -= hq;
      int64_t row = token;
      if (p.cache_rows != nullptr) {
        row = p.cache_rows[token];
        if (row < 0 || row >= p.num_rows) {  // a padded token's key and value go nowhere
          if (row >= p.num_rows) record_device_error(GDN_ERR_EXTENT);
          continue;
        }
      }
      value = h >= hk;
      if (value) h -= hk;
      x = value ? static_cast<const T*>(p.v) + token * p.v_stride : static_cast<const T*>(p.k) + token * p.k_stride;
      y = value ? static_cast<T*>(p.v_out) + row * p.v_out_stride : static_cast<T*>(p.k_out) + row * p.k_out_stride;
    }
    x += h * p.D;
    y += h * p.D;
    const bool turns = w < sh.turn;
    if (VECTOR) {
      if (HALF) {
        const int at = turns ? w * V : 2 * pairs + (w - sh.turn) * V;
        const Vec<T> a = *reinterpret_cast<const Vec<T>*>(x + at);
        if (!turns) {
          *reinterpret_cast<Vec<T>*>(y + at) = a;
          continue;
        }
        const Vec<T> b = *reinterpret_cast<const Vec<T>*>(x + at + pairs);
        Vec<T> ya = a, yb = b;
        if (!value) {
#pragma unroll
          for (int e = 0; e < V; ++e) {
            const float2 f = cs[t][at + e];
            const float x1 = to_f32(a.e[e]), x2 = to_f32(b.e[e]);
            ya.e[e] = from_f32<T>(x1 * f.x - x2 * f.y);
            yb.e[e] = from_f32<T>(x2 * f.x + x1 * f.y);
          }
        }
        *reinterpret_cast<Vec<T>*>(y + at) = ya;
        *reinterpret_cast<Vec<T>*>(y + at + pairs) = yb;
      } else {
        const int at = w * V;
        Vec<T> a = *reinterpret_cast<const Vec<T>*>(x + at);
        if (!value) {
#pragma unroll
          for (int e = 0; e < V; e += 2)
            if ((at + e) / 2 < pairs) {
              const float2 f = cs[t][(at + e) / 2];
              const float x1 = to_f32(a.e[e]), x2 = to_f32(a.e[e + 1]);
              a.e[e] = from_f32<T>(x1 * f.x - x2 * f.y);
              a.e[e + 1] = from_f32<T>(x2 * f.x + x1 * f.y);
            }
        }
        *reinterpret_cast<Vec<T>*>(y + at) = a;
      }
    } else {
      if (!turns) {
        y[2 * pairs + w - sh.turn] = x[2 * pairs + w - sh.turn];
        continue;
      }
      const T a = x[w], b = x[w + pairs];
      if (value) {
        y[w] = a;
        y[w + pairs] = b;
        continue;
      }
      const float2 f = cs[t][w];
      const float x1 = to_f32(a), x2 = to_f32(b);
      y[w] = from_f32<T>(x1 * f.x - x2 * f.y);
      y[w + pairs] = from_f32<T>(x2 * f.x + x1 * f.y);
    }
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
  // a CTA has two units a thread, or as many as there are where tokens are few
  const int64_t units = (int64_t)heads * (sh.turn + sh.copy);
  int64_t tokens = 2 * kRThreads / units;
  tokens = tokens < 1 ? 1 : tokens > kRMaxTokens ? kRMaxTokens : tokens;
  while (tokens > 1 && (p.T + tokens - 1) / tokens < 304) tokens /= 2;
  sh.tokens = (int)tokens;
  const int64_t ctas = (p.T + tokens - 1) / tokens;
  // few tokens: the heads of one over several CTAs
  int64_t parts = 1;
  while (parts < 8 && ctas * parts < 152 && units * tokens > parts * kRThreads) parts *= 2;
  const dim3 grid((unsigned)ctas, (unsigned)parts);
  if (!half) rope_kernel<T, false, true><<<grid, kRThreads, 0, stream>>>(p, sh);
  else if (vector) rope_kernel<T, true, true><<<grid, kRThreads, 0, stream>>>(p, sh);
  else rope_kernel<T, true, false><<<grid, kRThreads, 0, stream>>>(p, sh);
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
