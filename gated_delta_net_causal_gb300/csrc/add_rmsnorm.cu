// Residual addition, RMSNorm and quantisation of rows in one pass:
//   s = round(x + r);  y = s (mean s^2 + eps)^(-1/2) w;
//   out = round(y);  out_scale = max(max|y| / 448, 2^-126), out_q = e4m3(y / out_scale)
// s is rounded to the io dtype first, as the residual stream stores it, and
// the norm is taken of the stored values. The mean and the maximum are held
// in fp32. With t = s w, max|y| is max|t| times the inverse root, so both
// reductions of a row go through one barrier and its values stay in
// registers between: x and r are read once, each output is written once.
// Bound by those bytes: 8192 rows of 8192 bf16 with a residual to e4m3, 81 us,
// 5.8 TB/s (a copy: 6.8; one row a CTA without the ring below: 122 us); 999
// rows of 2051 fp16, which allow no wide accesses, 10.2 us.
#include <type_traits>

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

// x, y to two e4m3 codes (x in the low byte), nearest with ties to even
__device__ __forceinline__ uint32_t e4m3x2(float x, float y) {
  uint16_t r;
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(r) : "f"(y), "f"(x));
  return r;
}

// what the values of a row become once its reductions are there
struct RowScale {
  float inv, scale, inv_scale;
};
__device__ __forceinline__ RowScale row_scale(const AddRmsNormArgs& p, float ss, float top) {
  RowScale r;
  r.inv = p.norm_w == nullptr ? 1.f : 1.f / sqrtf(ss / (float)p.cols + p.eps);
  r.scale = fmaxf(top * r.inv / kE4m3Max, kScaleFloor);
  r.inv_scale = 1.f / r.scale;  // not inv / scale: a row of zeros would make that infinite
  return r;
}
// Elements 2 k and 2 k + 1 of a vector in fp32 (the second is 0 where VEC is 1)
template <int VEC>
__device__ __forceinline__ float2 pair(const Pack<float, VEC>& a, int k) {
  return make_float2(a.v[2 * k], VEC > 1 ? a.v[VEC > 1 ? 2 * k + 1 : 0] : 0.f);
}
template <int VEC>
__device__ __forceinline__ float2 pair(const Pack<__half, VEC>& a, int k) {
  if constexpr (VEC == 1) return make_float2(__half2float(a.v[0]), 0.f);
  else return __half22float2(reinterpret_cast<const __half2*>(a.v)[k]);
}
template <int VEC>
__device__ __forceinline__ float2 pair(const Pack<__nv_bfloat16, VEC>& a, int k) {
  if constexpr (VEC == 1) return make_float2(__bfloat162float(a.v[0]), 0.f);
  const uint32_t u = reinterpret_cast<const uint32_t*>(a.v)[VEC == 1 ? 0 : k];
  return make_float2(__uint_as_float(u << 16), __uint_as_float(u & 0xffff0000u));
}
// a + b rounded to T, two elements an instruction where T has 16 bits
template <int VEC>
__device__ __forceinline__ Pack<float, VEC> add(const Pack<float, VEC>& a, const Pack<float, VEC>& b) {
  Pack<float, VEC> c;
#pragma unroll
  for (int e = 0; e < VEC; ++e) c.v[e] = a.v[e] + b.v[e];
  return c;
}
template <typename T, int VEC>
__device__ __forceinline__ Pack<T, VEC> add(const Pack<T, VEC>& a, const Pack<T, VEC>& b) {
  Pack<T, VEC> c;
  if constexpr (VEC == 1) {
    c.v[0] = __hadd(a.v[0], b.v[0]);
  } else {
    using T2 = typename std::conditional<std::is_same<T, __half>::value, __half2, __nv_bfloat162>::type;
#pragma unroll
    for (int k = 0; k < VEC / 2; ++k)
      reinterpret_cast<T2*>(c.v)[k] = __hadd2(reinterpret_cast<const T2*>(a.v)[k], reinterpret_cast<const T2*>(b.v)[k]);
  }
  return c;
}
// weights of vector i (1 without)
template <int VEC>
struct Weights {
  float2 v[(VEC + 1) / 2];
};
template <int VEC>
__device__ __forceinline__ Weights<VEC> weights(const AddRmsNormArgs& p, int i) {
  Weights<VEC> w;
#pragma unroll
  for (int k = 0; k < (VEC + 1) / 2; ++k) w.v[k] = make_float2(1.f, 1.f);
  if (p.norm_w == nullptr) return w;
  if constexpr (VEC == 1) {
    w.v[0].x = __ldg(p.norm_w + i);
  } else {
#pragma unroll
    for (int e = 0; e < VEC; e += 4) {
      const float4 x = __ldg(reinterpret_cast<const float4*>(p.norm_w + (int64_t)i * VEC + e));
      w.v[e / 2] = make_float2(x.x, x.y);
      w.v[e / 2 + 1] = make_float2(x.z, x.w);
    }
  }
  return w;
}
__device__ __forceinline__ float2 times(float2 a, float2 b) { return fma2(a, b, make_float2(-0.f, -0.f)); }
// squares of s, and the maximum of |s w|
template <typename T, int VEC>
__device__ __forceinline__ void weigh(const Pack<T, VEC>& s, const Weights<VEC>& w, float2& ss, float& top) {
#pragma unroll
  for (int k = 0; k < (VEC + 1) / 2; ++k) {
    const float2 x = pair<VEC>(s, k);
    const float2 t = times(x, w.v[k]);
    ss = fma2(x, x, ss);
    top = fmaxf(top, fmaxf(fabsf(t.x), fabsf(t.y)));
  }
}
// vector i of the outputs of a row, from s
template <typename T, int VEC>
__device__ __forceinline__ void give(const AddRmsNormArgs& p, int64_t row, int i, const Pack<T, VEC>& s,
                                     const Weights<VEC>& w, const RowScale& r) {
  constexpr int N2 = (VEC + 1) / 2;
  float2 t[N2];
#pragma unroll
  for (int k = 0; k < N2; ++k) t[k] = times(times(pair<VEC>(s, k), w.v[k]), make_float2(r.inv, r.inv));
  if (p.out != nullptr) {
    Pack<T, VEC> c;
#pragma unroll
    for (int k = 0; k < N2; ++k) {
      c.v[2 * k] = from_f32<T>(t[k].x);
      if (VEC > 1) c.v[VEC > 1 ? 2 * k + 1 : 0] = from_f32<T>(t[k].y);
    }
    reinterpret_cast<Pack<T, VEC>*>(static_cast<T*>(p.out) + row * p.out_stride)[i] = c;
  }
  if (p.out_q != nullptr) {
    uint32_t q[N2];
#pragma unroll
    for (int k = 0; k < N2; ++k) {
      const float2 y = times(t[k], make_float2(r.inv_scale, r.inv_scale));
      q[k] = e4m3x2(y.x, y.y);
    }
    uint8_t* oq = static_cast<uint8_t*>(p.out_q) + row * p.out_q_stride + (int64_t)i * VEC;
    if constexpr (VEC == 8) *reinterpret_cast<uint2*>(oq) = make_uint2(q[0] | q[1] << 16, q[2] | q[3] << 16);
    else if constexpr (VEC == 4) *reinterpret_cast<uint32_t*>(oq) = q[0] | q[1] << 16;
    else *oq = (uint8_t)q[0];
  }
}
// sum of ss and maximum of top over the NT threads of a row; buf: its own for
// two rows in turn, so that one barrier a row is enough
template <int NT>
__device__ __forceinline__ void reduce_row(float2 ss2, float& ss, float& top, float (&buf)[2][32], int tid) {
  ss = group_sum<32>(ss2.x + ss2.y);
#pragma unroll
  for (int d = 16; d > 0; d >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, d));
  if (NT > 32) {
    if ((tid & 31) == 0) {
      buf[0][tid >> 5] = ss;
      buf[1][tid >> 5] = top;
    }
    __syncthreads();
    ss = 0.f;
    top = 0.f;
#pragma unroll
    for (int w = 0; w < NT / 32; ++w) {
      ss += buf[0][w];
      top = fmaxf(top, buf[1][w]);
    }
  }
}

// One row for NT threads (NT = 32: a warp, eight rows per CTA), for few rows
// and for rows that do not allow 16-byte accesses: thread t holds the NV
// vectors t, t + NT, ... in registers, all its loads issued before the first
// store. Rows longer than NT * NV * VEC go through their tail twice (REST).
template <typename T, int VEC, int NT, int NV, bool REST>
__global__ void __launch_bounds__(NT == 32 ? 256 : NT) add_rmsnorm_kernel(const AddRmsNormArgs p) {
  constexpr int ROWS = NT == 32 ? 8 : 1;
  const int tid = NT == 32 ? (threadIdx.x & 31) : threadIdx.x;
  const int64_t row = (int64_t)blockIdx.x * ROWS + (NT == 32 ? (threadIdx.x >> 5) : 0);
  if (row >= p.rows) return;
  using P = Pack<T, VEC>;
  __shared__ float red[2][32];
  const P* x = reinterpret_cast<const P*>(static_cast<const T*>(p.x) + row * p.x_stride);
  const P* r = p.residual == nullptr
                   ? nullptr
                   : reinterpret_cast<const P*>(static_cast<const T*>(p.residual) + row * p.residual_stride);
  P* sum = p.sum == nullptr ? nullptr : reinterpret_cast<P*>(static_cast<T*>(p.sum) + row * p.sum_stride);
  const int nvec = (int)(p.cols / VEC);
  float2 ss2 = make_float2(0.f, 0.f);
  float ss, top = 0.f;
  P a[NV];
  {
    P b[NV];
#pragma unroll
    for (int n = 0; n < NV; ++n)
      if (tid + n * NT < nvec) {
        a[n] = x[tid + n * NT];
        if (r != nullptr) b[n] = r[tid + n * NT];
      }
#pragma unroll
    for (int n = 0; n < NV; ++n) {
      const int i = tid + n * NT;
      if (i < nvec) {
        if (r != nullptr) a[n] = add(a[n], b[n]);
        if (sum != nullptr) sum[i] = a[n];
        weigh<T, VEC>(a[n], weights<VEC>(p, i), ss2, top);
      }
    }
  }
  if (REST)
    for (int i = tid + NV * NT; i < nvec; i += NT) {
      P s = x[i];
      if (r != nullptr) s = add(s, r[i]);
      if (sum != nullptr) sum[i] = s;
      weigh<T, VEC>(s, weights<VEC>(p, i), ss2, top);
    }
  reduce_row<NT>(ss2, ss, top, red, tid);
  const RowScale sc = row_scale(p, ss, top);
  if (p.out_q != nullptr && tid == 0) p.out_scale[row] = sc.scale;
#pragma unroll
  for (int n = 0; n < NV; ++n)
    if (tid + n * NT < nvec) give<T, VEC>(p, row, tid + n * NT, a[n], weights<VEC>(p, tid + n * NT), sc);
  if (REST)
    for (int i = tid + NV * NT; i < nvec; i += NT) {
      // the sum as stored: it may be where x or the residual was
      P s = sum != nullptr ? sum[i] : x[i];
      if (r != nullptr && sum == nullptr) s = add(s, r[i]);
      give<T, VEC>(p, row, i, s, weights<VEC>(p, i), sc);
    }
}

// Many rows: as many CTAs as the SMs hold, each with a ring of rows of x and
// the residual that bulk copies fill ahead, so that the memory is read while
// rows are reduced and stored. A thread keeps its columns' weights for all of
// its rows, and its part of a row between the two passes. The barrier of a
// row's reduction is also the one after which its place is filled again.
constexpr int kRingSlots = 8;

template <typename T, int NT, int NV>
__global__ void __launch_bounds__(NT) add_rmsnorm_ring_kernel(const AddRmsNormArgs p, const int slots) {
  constexpr int VEC = 16 / sizeof(T);
  using P = Pack<T, VEC>;
  extern __shared__ __align__(128) unsigned char ring[];
  __shared__ __align__(8) uint64_t full[kRingSlots];
  __shared__ float red[2][2][32];
  __shared__ int s_abort;
  const int tid = threadIdx.x;
  const uint32_t bytes = (uint32_t)p.cols * sizeof(T), slot_bytes = p.residual == nullptr ? bytes : 2 * bytes;
  const int nvec = (int)(p.cols / VEC);
  if (tid == 0) {
    for (int s = 0; s < slots; ++s) mbar_init(&full[s], 1);
    s_abort = 0;
    fence_mbar_init();
  }
  __syncthreads();
  volatile int* abort_flag = &s_abort;
  const auto fill = [&](int s, int64_t row) {
    mbar_arrive_expect_tx(&full[s], slot_bytes);
    bulk_load(ring + (size_t)s * slot_bytes, static_cast<const T*>(p.x) + row * p.x_stride, bytes, &full[s]);
    if (p.residual != nullptr)
      bulk_load(ring + (size_t)s * slot_bytes + bytes, static_cast<const T*>(p.residual) + row * p.residual_stride, bytes,
                &full[s]);
  };
  int64_t fills = 0;  // thread 0's
  if (tid == 0)
    for (; fills < slots && blockIdx.x + fills * gridDim.x < p.rows; ++fills)
      fill((int)fills, blockIdx.x + fills * gridDim.x);
  Weights<VEC> w[NV];
#pragma unroll
  for (int n = 0; n < NV; ++n)
    if (tid + n * NT < nvec) w[n] = weights<VEC>(p, tid + n * NT);
  int slot = 0, parity = 0;
  uint32_t phase = 0;
  for (int64_t row = blockIdx.x; row < p.rows; row += gridDim.x, parity ^= 1) {
    const bool ok = mbar_wait_bounded(&full[slot], phase, abort_flag);
    const P* x = reinterpret_cast<const P*>(ring + (size_t)slot * slot_bytes);
    P* sum = p.sum == nullptr ? nullptr : reinterpret_cast<P*>(static_cast<T*>(p.sum) + row * p.sum_stride);
    float2 ss2 = make_float2(0.f, 0.f);
    float ss, top = 0.f;
    P a[NV];
#pragma unroll
    for (int n = 0; n < NV; ++n) {
      const int i = tid + n * NT;
      if (i < nvec && ok) {
        a[n] = x[i];
        if (p.residual != nullptr) a[n] = add(a[n], x[nvec + i]);
        if (sum != nullptr) sum[i] = a[n];
        weigh<T, VEC>(a[n], w[n], ss2, top);
      }
    }
    reduce_row<NT>(ss2, ss, top, red[parity], tid);
    // every thread has read the row
    if (tid == 0 && !*abort_flag) {
      const int64_t next = row + (int64_t)slots * gridDim.x;
      if (next < p.rows) {
        fill(slot, next);
        ++fills;
      }
    }
    if (ok) {
      const RowScale sc = row_scale(p, ss, top);
      if (p.out_q != nullptr && tid == 0) p.out_scale[row] = sc.scale;
#pragma unroll
      for (int n = 0; n < NV; ++n)
        if (tid + n * NT < nvec) give<T, VEC>(p, row, tid + n * NT, a[n], w[n], sc);
    }
    if (++slot == slots) {
      slot = 0;
      phase ^= 1;
    }
  }
  // after a wait that gave up: no copy may be in flight when the CTA ends
  if (tid == 0 && *abort_flag)
    for (int s = 0; s < slots && s < fills; ++s) mbar_wait(&full[s], ((fills - s + slots - 1) / slots - 1) & 1);
}

int norm_sms() {
  int dev = 0, n = 0;
  if (cudaGetDevice(&dev) != cudaSuccess ||
      cudaDeviceGetAttribute(&n, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess || n <= 0)
    return 148;
  return n;
}

template <typename T, int NT, int NV>
cudaError_t launch_ring(const AddRmsNormArgs& p, int ctas_per_sm, int slots, int64_t slot_bytes, cudaStream_t stream) {
  auto kern = add_rmsnorm_ring_kernel<T, NT, NV>;
  const int smem = (int)(slots * slot_bytes);
  const cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
  if (e != cudaSuccess) return e;
  kern<<<(unsigned)(ctas_per_sm * norm_sms()), NT, smem, stream>>>(p, slots);
  return cudaGetLastError();
}

template <typename T, int VEC, int NT, int NV, bool REST>
cudaError_t launch_norm_k(const AddRmsNormArgs& p, cudaStream_t stream) {
  constexpr int ROWS = NT == 32 ? 8 : 1;
  add_rmsnorm_kernel<T, VEC, NT, NV, REST>
      <<<(unsigned)((p.rows + ROWS - 1) / ROWS), NT == 32 ? 256 : NT, 0, stream>>>(p);
  return cudaGetLastError();
}

template <typename T, int VEC>
cudaError_t launch_norm_v(const AddRmsNormArgs& p, cudaStream_t stream) {
  const int64_t nvec = p.cols / VEC;
  if constexpr (VEC > 1) {
    // the ring where every CTA has rows enough to run ahead, and two of them fit
    const int64_t slot_bytes = p.cols * (int64_t)sizeof(T) * (p.residual == nullptr ? 1 : 2);
    const int per_sm = slot_bytes <= 36 * 1024 ? 3 : 2;
    int64_t slots = (per_sm == 3 ? 72 : 110) * 1024 / slot_bytes;
    if (slots > kRingSlots) slots = kRingSlots;
    if (nvec > 64 && nvec <= 2048 && slots >= 2 && p.rows >= 4ll * per_sm * norm_sms()) {
      const int n = (int)slots;
      if (nvec <= 128) return launch_ring<T, 128, 1>(p, per_sm, n, slot_bytes, stream);
      if (nvec <= 256) return launch_ring<T, 256, 1>(p, per_sm, n, slot_bytes, stream);
      if (nvec <= 512) return launch_ring<T, 256, 2>(p, per_sm, n, slot_bytes, stream);
      if (nvec <= 1024) return launch_ring<T, 256, 4>(p, per_sm, n, slot_bytes, stream);
      return launch_ring<T, 512, 4>(p, per_sm, n, slot_bytes, stream);
    }
  }
  if (nvec <= 64) return launch_norm_k<T, VEC, 32, 2, false>(p, stream);
  if (nvec <= 256) return launch_norm_k<T, VEC, 128, 2, false>(p, stream);
  if (nvec <= 512) return launch_norm_k<T, VEC, 256, 2, false>(p, stream);
  if (nvec <= 1024) return launch_norm_k<T, VEC, 256, 4, false>(p, stream);
  if (nvec <= 2048) return launch_norm_k<T, VEC, 512, 4, false>(p, stream);
  if (VEC == 1 && nvec <= 4096) return launch_norm_k<T, VEC, 512, VEC == 1 ? 8 : 4, false>(p, stream);
  return launch_norm_k<T, VEC, 512, 4, true>(p, stream);
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

GDN_DEFINE_ERROR_READER(add_rmsnorm)
