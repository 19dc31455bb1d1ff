// Puts the parts of softmax attention together, and chooses the kernels.
//
// attn_join_kernel: block (b, y) looks whether CTA b of the attention kernel
// ended its stretch within an item; the parts of that item are then its last
// one, those of the CTAs after it that had nothing else, and the first one of
// the CTA that ended it. A warp takes a row: the largest score of the parts,
// their factors, and the sum of the parts' outputs, always in CTA order. Bound
// by memory's latency, a wave of CTAs after the other: about 8 us for the 40 MB
// of parts of a prompt, 4 us for a single token's. (At head_dim 128 it has
// 32 registers and 4 bytes spilled.)
#include "attn_common.cuh"

namespace gdn {
namespace {

constexpr int kJWarps = 8;

// four elements of a row times f, in fp32 where there is a place for that
template <typename T>
__device__ __forceinline__ void put_row(void* out, float* wide, int64_t at, float f, float4 o) {
  o = make_float4(o.x * f, o.y * f, o.z * f, o.w * f);
  if (wide != nullptr) {
    *reinterpret_cast<float4*>(wide + at) = o;
  } else {
    T* y = static_cast<T*>(out) + at;
    y[0] = from_f32<T>(o.x), y[1] = from_f32<T>(o.y), y[2] = from_f32<T>(o.z), y[3] = from_f32<T>(o.w);
  }
}

template <typename T, int D>
__global__ void __launch_bounds__(32 * kJWarps) attn_join_kernel(const AttnArgs p, int ctas) {
  grid_dependency_wait();
  const int b = blockIdx.x, lane = threadIdx.x & 31;
  const int r = blockIdx.y * kJWarps + (threadIdx.x >> 5);
  // part j of the item: what CTA b ended with, then what CTA b + j began with;
  // lane j looks at it (and at its row) before it is known to be one, so that
  // the loads wait for memory together
  const auto slot_of = [&](int j) { return (int64_t)(j == 0 ? 2 * b + 1 : 2 * (b + j)); };
  const int4 at = p.part_at[2 * b + 1];
  const bool in = b + lane < ctas;
  const int4 mine = in ? p.part_at[slot_of(lane)] : make_int4(0, 0, 0, 0);
  float2 ml = in && r < p.part_rows ? p.part_ml[slot_of(lane) * p.part_rows + r] : make_float2(0.f, 0.f);
  if ((at.x & 3) != kAttnFirst || r >= at.z * p.group) return;
  unsigned end = __ballot_sync(0xffffffffu, (mine.x & 3) == kAttnLast && lane > 0);
  int parts = end != 0 ? __ffs(end) : 0;
  for (int j0 = 32; parts == 0; j0 += 32) {  // more than 32 parts
    if (b + j0 >= ctas) return;              // (an item that is begun is ended)
    end = __ballot_sync(0xffffffffu, b + j0 + lane < ctas && (p.part_at[slot_of(j0 + lane)].x & 3) == kAttnLast);
    if (end != 0) parts = j0 + __ffs(end);
  }
  const int64_t token = at.y + r / p.group;
  const int head = attn_head(p, at.w, r % p.group);
  float top = lane < parts ? ml.x : -INFINITY;
  for (int j = lane + 32; j < parts; j += 32) top = fmaxf(top, p.part_ml[slot_of(j) * p.part_rows + r].x);
#pragma unroll
  for (int d = 16; d > 0; d >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, d));
  const float base = top == -INFINITY ? 0.f : top;
  const bool holds = 4 * lane < D;
  float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
  float sum = 0.f;
  for (int j0 = 0; j0 < parts; j0 += 32) {
    if (j0 > 0 && j0 + lane < parts) ml = p.part_ml[slot_of(j0 + lane) * p.part_rows + r];
    float f = 0.f;
    if (j0 + lane < parts) {
      f = exp2f(ml.x - base);
      sum = fmaf(ml.y, f, sum);
    }
    const int n = parts - j0 < 32 ? parts - j0 : 32;
#pragma unroll 1
    for (int j1 = 0; j1 < n; j1 += 8) {
      float4 x[8];
#pragma unroll
      for (int j = 0; j < 8; ++j)
        x[j] = holds && j1 + j < n ? *reinterpret_cast<const float4*>(
                                         p.part_o + (slot_of(j0 + j1 + j) * p.part_rows + r) * D + 4 * lane)
                                   : make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        // (a part without keys has the factor 0 and zeros)
        const float w = __shfl_sync(0xffffffffu, f, (j1 + j) & 31);
        o.x = fmaf(w, x[j].x, o.x), o.y = fmaf(w, x[j].y, o.y), o.z = fmaf(w, x[j].z, o.z), o.w = fmaf(w, x[j].w, o.w);
      }
    }
  }
  sum = group_sum<32>(sum);
  const int causal = at.x >> 2;
  float* lse = attn_lse(p, causal);
  float* part_out = attn_part_out(p, causal);
  const AttnScale f = attn_scale(top, sum, lse != nullptr);
  if (holds) put_row<T>(p.out, part_out, (token * p.Hq + head) * D + 4 * lane, f.factor, o);
  if (lane == 0 && lse != nullptr) lse[token * p.Hq + head] = f.lse;
}

// With groups: a row's outputs over its own keys and over its group's prefix,
// by their sums. A warp a row.
template <typename T, int D>
__global__ void __launch_bounds__(32 * kJWarps) attn_merge_kernel(const AttnArgs p) {
  grid_dependency_wait();
  const int lane = threadIdx.x & 31;
  const int64_t row = (int64_t)blockIdx.x * kJWarps + (threadIdx.x >> 5), token = row / p.Hq;
  if (token >= p.T || token < p.cu_seqlens[0] || token >= p.cu_seqlens[p.N]) return;  // no sequence's
  const bool any = token >= p.group_cu[0] && token < p.group_cu[p.groups];
  const float a = p.part_lse[0][row], b = any ? p.part_lse[1][row] : -INFINITY;
  const bool holds = 4 * lane < D;
  const float4 zero = make_float4(0.f, 0.f, 0.f, 0.f);
  const float4 x = holds ? *reinterpret_cast<const float4*>(p.part_out[0] + row * D + 4 * lane) : zero;
  const float4 y = holds && any ? *reinterpret_cast<const float4*>(p.part_out[1] + row * D + 4 * lane) : zero;
  float m = fmaxf(a, b);
  if (m == -INFINITY) m = 0.f;  // nothing is seen
  const float wa = expf(a - m), wb = expf(b - m), s = wa + wb;
  const float inv = s == 0.f ? 0.f : 1.f / s, fa = wa * inv, fb = wb * inv;
  if (holds)
    put_row<T>(p.out, nullptr, row * D + 4 * lane, 1.f,
               make_float4(fmaf(fa, x.x, fb * y.x), fmaf(fa, x.y, fb * y.y), fmaf(fa, x.z, fb * y.z),
                           fmaf(fa, x.w, fb * y.w)));
  if (lane == 0 && p.lse != nullptr) p.lse[row] = s == 0.f ? -INFINITY : m + logf(s);
}

// Their launches overlap the end of the kernel before (all of them wait for it).
template <typename... A>
cudaError_t launch_after(void (*kernel)(A...), dim3 grid, cudaStream_t stream, A... args) {
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = grid;
  cfg.blockDim = dim3(32 * kJWarps);
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kernel, args...);
}
template <typename T, int D>
cudaError_t join(const AttnArgs& p, int ctas, cudaStream_t stream) {
  if (p.part_o != nullptr) {
    const dim3 grid((unsigned)ctas, (unsigned)((p.part_rows + kJWarps - 1) / kJWarps));
    const cudaError_t e = launch_after(attn_join_kernel<T, D>, grid, stream, p, ctas);
    if (e != cudaSuccess) return e;
  }
  if (p.groups == 0) return cudaSuccess;
  const int64_t rows = (int64_t)p.T * p.Hq;
  return launch_after(attn_merge_kernel<T, D>, dim3((unsigned)((rows + kJWarps - 1) / kJWarps)), stream, p);
}
template <typename T>
cudaError_t join_dim(const AttnArgs& p, int32_t D, int ctas, cudaStream_t stream) {
  switch (D) {
    case 32: return join<T, 32>(p, ctas, stream);
    case 64: return join<T, 64>(p, ctas, stream);
    case 96: return join<T, 96>(p, ctas, stream);
    default: return join<T, 128>(p, ctas, stream);
  }
}

int sm_count() {
  int dev = 0, n = 0;
  if (cudaGetDevice(&dev) != cudaSuccess ||
      cudaDeviceGetAttribute(&n, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess || n <= 0)
    return 152;
  return n;
}

int64_t round256(int64_t n) { return (n + 255) / 256 * 256; }

}  // namespace

AttnSplit attn_split(int32_t dtype, int64_t T, int32_t group, int32_t D) {
  AttnSplit s{};
  if (dtype == GDN_F32) {
    s.ctas = attn_cc_ctas(sm_count());
    s.item = attn_cc_rows() / group;
  } else {
    s.ctas = sm_count();
    s.item = 2 * (attn_tc_rows() / group);
  }
  s.rows = (int32_t)(T < s.item ? T : s.item) * group;
  const int64_t slots = 2ll * s.ctas;
  s.ml_at = round256(slots * s.rows * D * 4);
  s.at_at = s.ml_at + round256(slots * s.rows * 8);
  s.bytes = s.at_at + round256(slots * 16);
  return s;
}

cudaError_t launch_attn(AttnArgs p, const AttnSplit& s, void* workspace, int32_t dtype, int32_t D,
                        cudaStream_t stream) {
  p.item = s.item;
  p.part_rows = s.rows;
  char* ws = static_cast<char*>(workspace);
  if (ws != nullptr) {
    p.part_o = reinterpret_cast<float*>(ws);
    p.part_ml = reinterpret_cast<float2*>(ws + s.ml_at);
    p.part_at = reinterpret_cast<int4*>(ws + s.at_at);
  }
  const cudaError_t e = dtype == GDN_F32 ? launch_attn_cc(p, D, s.ctas, stream)
                                         : launch_attn_tc(p, dtype, D, s.ctas, stream);
  if (e != cudaSuccess || ws == nullptr) return e;
  switch (dtype) {
    case GDN_F16: return join_dim<__half>(p, D, s.ctas, stream);
    case GDN_BF16: return join_dim<__nv_bfloat16>(p, D, s.ctas, stream);
    default: return join_dim<float>(p, D, s.ctas, stream);
  }
}

}  // namespace gdn
