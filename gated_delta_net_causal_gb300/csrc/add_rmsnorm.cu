// Residual addition, RMSNorm and quantisation of rows in one pass:
//   s = round(x + r);  y = s (mean s^2 + eps)^(-1/2) w;
//   out = round(y);  out_scale = max(max|y| / 448, 2^-126), out_q = e4m3(y / out_scale)
// s is rounded to the io dtype first, as the residual stream stores it, and
// the norm is taken of the stored values. The mean and the maximum are held
// in fp32. With t = s w, max|y| is max|t| times the inverse root, so both
// reductions of a row go through one barrier and its values stay in
// registers between: x and r are read once, each output is written once.
#include <cuda_fp8.h>

#include "gdn_common.cuh"
#include "gdn_internal.h"

namespace gdn {
namespace {

constexpr float kE4m3Max = 448.f;
constexpr float kScaleFloor = 1.17549435e-38f;  // 2^-126: its inverse is finite, and a zero row's codes are 0

template <typename T, int VEC>
struct Pack;  // VEC elements of T as one access
template <typename T>
struct alignas(sizeof(T)) Pack<T, 1> {
  T v[1];
};
template <typename T>
struct alignas(16) Pack<T, 4> {
  T v[4];
};
template <typename T>
struct alignas(16) Pack<T, 8> {
  T v[8];
};

__device__ __forceinline__ uint8_t e4m3(float x) {
  return (uint8_t)__nv_cvt_float_to_fp8(x, __NV_SATFINITE, __NV_E4M3);
}

// One CTA of NT threads per row (NT = 32: one warp per row, eight rows per
// CTA). Thread t holds the NV vectors t, t + NT, ... of its row; rows longer
// than NT * NV * VEC go through their tail twice (REST).
template <typename T, int VEC, int NT, int NV, bool REST>
__global__ void __launch_bounds__(NT == 32 ? 256 : NT) add_rmsnorm_kernel(const AddRmsNormArgs p) {
  constexpr int ROWS = NT == 32 ? 8 : 1;
  const int tid = NT == 32 ? (threadIdx.x & 31) : threadIdx.x;
  const int64_t row = (int64_t)blockIdx.x * ROWS + (NT == 32 ? (threadIdx.x >> 5) : 0);
  if (row >= p.rows) return;
  using P = Pack<T, VEC>;
  const T* x = static_cast<const T*>(p.x) + row * p.x_stride;
  const T* r = p.residual == nullptr ? nullptr : static_cast<const T*>(p.residual) + row * p.residual_stride;
  T* sum = p.sum == nullptr ? nullptr : static_cast<T*>(p.sum) + row * p.sum_stride;
  const int nvec = (int)(p.cols / VEC);

  float ss = 0.f, top = 0.f;
  // s = x (+ residual) of vector i, stored; read back the second time (sum may
  // be the residual itself)
  auto load = [&](int i, P& a, P& b, bool again) {
    const bool stored = again && sum != nullptr;
    a = *reinterpret_cast<const P*>((stored ? sum : x) + (int64_t)i * VEC);
    if (r != nullptr && !stored) b = *reinterpret_cast<const P*>(r + (int64_t)i * VEC);
  };
  // t = s w, and the first time its squares and maximum
  auto take = [&](int i, const P& a, const P& b, float (&t)[VEC], bool again) {
    P c = a;
    if (r != nullptr && !(again && sum != nullptr))
#pragma unroll
      for (int e = 0; e < VEC; ++e) c.v[e] = from_f32<T>(to_f32(a.v[e]) + to_f32(b.v[e]));
    if (sum != nullptr && !again) *reinterpret_cast<P*>(sum + (int64_t)i * VEC) = c;
    alignas(16) float w[VEC];
    if (p.norm_w == nullptr) {
#pragma unroll
      for (int e = 0; e < VEC; ++e) w[e] = 1.f;
    } else if constexpr (VEC % 4 == 0) {
#pragma unroll
      for (int e = 0; e < VEC; e += 4)
        *reinterpret_cast<float4*>(w + e) = __ldg(reinterpret_cast<const float4*>(p.norm_w + (int64_t)i * VEC + e));
    } else {
      w[0] = __ldg(p.norm_w + i);
    }
#pragma unroll
    for (int e = 0; e < VEC; ++e) {
      const float s = to_f32(c.v[e]);
      if (!again) ss = fmaf(s, s, ss);
      t[e] = s * w[e];
      if (!again) top = fmaxf(top, fabsf(t[e]));
    }
  };
  // all of the row's loads before the first store, which they might not pass
  float t[NV][VEC];
  {
    P a[NV], b[NV];
#pragma unroll
    for (int n = 0; n < NV; ++n)
      if (tid + n * NT < nvec) load(tid + n * NT, a[n], b[n], false);
#pragma unroll
    for (int n = 0; n < NV; ++n)
      if (tid + n * NT < nvec) take(tid + n * NT, a[n], b[n], t[n], false);
  }
  if (REST)
    for (int i = tid + NV * NT; i < nvec; i += NT) {
      P a, b;
      float u[VEC];
      load(i, a, b, false);
      take(i, a, b, u, false);
    }

  ss = group_sum<32>(ss);
#pragma unroll
  for (int d = 16; d > 0; d >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, d));
  if (NT > 32) {
    __shared__ float red[2][32];
    if ((tid & 31) == 0) {
      red[0][tid >> 5] = ss;
      red[1][tid >> 5] = top;
    }
    __syncthreads();
    ss = 0.f;
    top = 0.f;
#pragma unroll
    for (int w = 0; w < NT / 32; ++w) {
      ss += red[0][w];
      top = fmaxf(top, red[1][w]);
    }
  }
  const float inv = p.norm_w == nullptr ? 1.f : 1.f / sqrtf(ss / (float)p.cols + p.eps);
  const float scale = fmaxf(top * inv / kE4m3Max, kScaleFloor);
  const float inv_q = inv / scale;
  T* out = p.out == nullptr ? nullptr : static_cast<T*>(p.out) + row * p.out_stride;
  uint8_t* oq = p.out_q == nullptr ? nullptr : static_cast<uint8_t*>(p.out_q) + row * p.out_q_stride;
  if (oq != nullptr && tid == 0) p.out_scale[row] = scale;
  auto give = [&](int i, const float (&u)[VEC]) {
    if (out != nullptr) {
      P c;
#pragma unroll
      for (int e = 0; e < VEC; ++e) c.v[e] = from_f32<T>(u[e] * inv);
      *reinterpret_cast<P*>(out + (int64_t)i * VEC) = c;
    }
    if (oq != nullptr) {
      uint8_t b[VEC];
#pragma unroll
      for (int e = 0; e < VEC; ++e) b[e] = e4m3(u[e] * inv_q);
      if constexpr (VEC == 8) {
        *reinterpret_cast<uint2*>(oq + (int64_t)i * VEC) = *reinterpret_cast<const uint2*>(b);
      } else if constexpr (VEC == 4) {
        *reinterpret_cast<uint32_t*>(oq + (int64_t)i * VEC) = *reinterpret_cast<const uint32_t*>(b);
      } else {
        oq[i] = b[0];
      }
    }
  };
#pragma unroll
  for (int n = 0; n < NV; ++n) {
    const int i = tid + n * NT;
    if (i < nvec) give(i, t[n]);
  }
  if (REST)
    for (int i = tid + NV * NT; i < nvec; i += NT) {
      P a, b;
      float u[VEC];
      load(i, a, b, true);
      take(i, a, b, u, true);
      give(i, u);
    }
}

template <typename T, int VEC>
cudaError_t launch_norm_v(const AddRmsNormArgs& p, cudaStream_t stream) {
  const int64_t nvec = p.cols / VEC;
  const unsigned rows = (unsigned)p.rows, rows8 = (unsigned)((p.rows + 7) / 8);
  if (nvec <= 64) add_rmsnorm_kernel<T, VEC, 32, 2, false><<<rows8, 256, 0, stream>>>(p);
  else if (nvec <= 256) add_rmsnorm_kernel<T, VEC, 128, 2, false><<<rows, 128, 0, stream>>>(p);
  else if (nvec <= 1024) add_rmsnorm_kernel<T, VEC, 256, 4, false><<<rows, 256, 0, stream>>>(p);
  else if (nvec <= 2048) add_rmsnorm_kernel<T, VEC, 512, 4, false><<<rows, 512, 0, stream>>>(p);
  else add_rmsnorm_kernel<T, VEC, 512, 4, true><<<rows, 512, 0, stream>>>(p);
  return cudaGetLastError();
}

template <typename T>
cudaError_t launch_norm_t(const AddRmsNormArgs& p, cudaStream_t stream) {
  constexpr int VEC = 16 / sizeof(T);
  // 16-byte accesses where every row of every tensor allows them
  auto fits = [](const void* ptr, int64_t stride, int64_t bytes) {
    return ptr == nullptr || (reinterpret_cast<uintptr_t>(ptr) % bytes == 0 && stride % VEC == 0);
  };
  if (p.cols % VEC == 0 && fits(p.x, p.x_stride, 16) && fits(p.residual, p.residual_stride, 16) &&
      fits(p.sum, p.sum_stride, 16) && fits(p.out, p.out_stride, 16) && fits(p.out_q, p.out_q_stride, VEC))
    return launch_norm_v<T, VEC>(p, stream);
  return launch_norm_v<T, 1>(p, stream);
}

}  // namespace

cudaError_t launch_add_rmsnorm(const AddRmsNormArgs& p, int32_t dtype, cudaStream_t stream) {
  if (p.rows == 0) return cudaSuccess;
  switch (dtype) {
    case GDN_F16: return launch_norm_t<__half>(p, stream);
    case GDN_BF16: return launch_norm_t<__nv_bfloat16>(p, stream);
    case GDN_F32: return launch_norm_t<float>(p, stream);
    default: return cudaErrorInvalidValue;
  }
}

}  // namespace gdn
