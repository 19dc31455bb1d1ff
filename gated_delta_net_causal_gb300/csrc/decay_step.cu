// One token of linear attention with a decay for each head, per sequence:
//   S = exp(g) S + v k^T,   o = scale S q,   optionally the gated RMSNorm of o.
// Bound by the fp32 state, read once and written once (128 KB per sequence
// and V head at D = 128). One CTA takes one (sequence, V head): every thread
// loads its whole share of the state (64 floats at D = 128) with 16-byte
// loads before it uses any, so a CTA has 64 KB in flight and the CTAs
// resident on an SM cover each other's compute and stores. The rows of a
// state are independent but for the norm, which takes one barrier.
// Measured: 128 sequences x 48 heads 119 us, 6.8 TB/s (a copy: 6.8); 64 rows of
// a pool, 32 heads, 44.5 us, 6.1 TB/s. States are read and written once: loads
// and stores marked so (ordinary stores: 125 and 47 us).
#include "decay_common.cuh"

namespace gdn {

template <typename T, int D>
__global__ void __launch_bounds__(DecayGeom<D>::THREADS) decay_step_kernel(const DecayArgs p) {
  using G = DecayGeom<D>;
  constexpr int LPR = G::LPR, NV4 = G::NV4, RPL = G::RPL, RPW = G::RPW;
  __shared__ float so[D];
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int sub = lane % LPR, rq = lane / LPR;
  const int h = blockIdx.x, b = blockIdx.y;
  const int kh = k_head_of(p.map, h, p.Hk, p.rep);
  int slot = b;
  if (p.slots != nullptr) {
    slot = p.slots[b];
    if (slot >= p.num_slots) {
      if (tid == 0 && h == 0) record_device_error(GDN_ERR_EXTENT);
      slot = -1;
    }
  }
  const int64_t orow = ((int64_t)b * p.Hv + h) * D;
  if (slot < 0) {  // a padded row: zero outputs, no state
    for (int j = tid; j < D; j += G::THREADS) {
      if (p.core_out != nullptr) p.core_out[orow + j] = 0.f;
      if (p.out != nullptr) static_cast<T*>(p.out)[orow + j] = from_f32<T>(0.f);
    }
    return;
  }
  float* S = p.state + ((int64_t)slot * p.Hv + h) * (int64_t)(D * D) + 4 * sub;
  float4 s[RPL][NV4];
#pragma unroll
  for (int u = 0; u < RPL; ++u)
#pragma unroll
    for (int m = 0; m < NV4; ++m)
      s[u][m] = __ldcs(reinterpret_cast<const float4*>(S + (warp * G::WROWS + u * RPW + rq) * D + 4 * LPR * m));
  const T* q = static_cast<const T*>(p.q) + (int64_t)b * p.q_stride + kh * D + 4 * sub;
  const T* k = static_cast<const T*>(p.k) + (int64_t)b * p.k_stride + kh * D + 4 * sub;
  const T* v = static_cast<const T*>(p.v) + (int64_t)b * p.v_stride + h * D;
  float4 qr[NV4], kr[NV4];
#pragma unroll
  for (int m = 0; m < NV4; ++m) {
    qr[m] = load4(q + 4 * LPR * m);
    kr[m] = load4(k + 4 * LPR * m);
  }
  float vr[RPL];
#pragma unroll
  for (int u = 0; u < RPL; ++u) vr[u] = to_f32(v[warp * G::WROWS + u * RPW + rq]);
  const Decay decay = decay_factor(decay_log(p.g[(int64_t)b * p.g_stride + h]));
  float o[RPL];
#pragma unroll
  for (int u = 0; u < RPL; ++u) {
    decay_update<NV4>(s[u], kr, decay, vr[u]);
    o[u] = row_dot<NV4>(s[u], qr);
    float* row = S + (warp * G::WROWS + u * RPW + rq) * D;
#pragma unroll
    for (int m = 0; m < NV4; ++m) __stcs(reinterpret_cast<float4*>(row + 4 * LPR * m), s[u][m]);
  }
#pragma unroll
  for (int d = LPR / 2; d > 0; d >>= 1)
#pragma unroll
    for (int u = 0; u < RPL; ++u) o[u] += __shfl_xor_sync(0xffffffffu, o[u], d);
  if (sub == 0)
#pragma unroll
    for (int u = 0; u < RPL; ++u) so[warp * G::WROWS + u * RPW + rq] = o[u] * p.scale;
  __syncthreads();
  if (warp == 0)
    decay_write_row<T, D>(so, p.core_out == nullptr ? nullptr : p.core_out + orow,
                          p.z == nullptr ? nullptr
                                         : static_cast<const T*>(p.z) + (int64_t)b * p.z_stride + h * D,
                          p.norm_w, p.out == nullptr ? nullptr : static_cast<T*>(p.out) + orow, p.rms_eps, lane);
}

template <typename T>
static cudaError_t launch_step_t(const DecayArgs& p, int32_t D, int32_t batch, cudaStream_t stream) {
  const dim3 grid((unsigned)p.Hv, (unsigned)batch);
  switch (D) {
    case 32: decay_step_kernel<T, 32><<<grid, DecayGeom<32>::THREADS, 0, stream>>>(p); break;
    case 64: decay_step_kernel<T, 64><<<grid, DecayGeom<64>::THREADS, 0, stream>>>(p); break;
    case 96: decay_step_kernel<T, 96><<<grid, DecayGeom<96>::THREADS, 0, stream>>>(p); break;
    case 128: decay_step_kernel<T, 128><<<grid, DecayGeom<128>::THREADS, 0, stream>>>(p); break;
    default: return cudaErrorInvalidValue;
  }
  return cudaGetLastError();
}

cudaError_t launch_decay_step(const DecayArgs& p, int32_t dtype, int32_t D, int32_t batch, cudaStream_t stream) {
  switch (dtype) {
    case GDN_F16: return launch_step_t<__half>(p, D, batch, stream);
    case GDN_BF16: return launch_step_t<__nv_bfloat16>(p, D, batch, stream);
    case GDN_F32: return launch_step_t<float>(p, D, batch, stream);
    default: return cudaErrorInvalidValue;
  }
}

}  // namespace gdn

GDN_DEFINE_ERROR_READER(decay_step)
