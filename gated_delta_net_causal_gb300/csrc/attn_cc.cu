// Softmax attention on the fp32 units (f32): rows x keys in tiles of 64 x 64, one
// pass over the keys with the running maximum and sum of each row.
//
// A CTA of 256 threads is a grid of 16 x 16; a thread has 4 x 4 scores (rows
// 4 ty + i, keys 4 tx + j), then the outputs of the same four rows at D / 16
// columns. q and k lie transposed in shared memory, so that a step of the
// contraction is two 16-byte reads for 16 products; the weights take k's
// place, transposed as well. Warps without a row (a single token has a few of
// the 64) only load. 4096 tokens, 8 / 2 heads of 128: 0.90 ms, 38 TFLOP/s, half
// of the fp32 units' rate; 32 tokens on up to 8192 keys, 32 / 8 heads, 479 us,
// 2.3 TB/s; 64 tokens behind 8192 shared keys 433 us. Bound by shared memory and
// by the phases between barriers: with one buffer, memory idles while a tile is
// computed, and the units while it is loaded.
#include "attn_common.cuh"

namespace gdn {
namespace {

constexpr int kAR = 64;    // rows of an item
constexpr int kAK = 64;    // keys of a tile
constexpr int kAT = 256;   // threads
constexpr int kAP = 68;    // pitch of the transposed tiles, in floats

// shared memory, in floats: q, k (whose place the weights take), v
template <int D>
struct CcSmem {
  static constexpr int kK = D * kAP, kV = kK + (D > kAK ? D : kAK) * kAP, kEnd = kV + kAK * D;
};

__device__ __forceinline__ float4 load4(const float* p) { return *reinterpret_cast<const float4*>(p); }
// four elements of a row, into a column of a transposed tile
__device__ __forceinline__ void put(float* t, float4 x) {
  t[0] = x.x, t[kAP] = x.y, t[2 * kAP] = x.z, t[3 * kAP] = x.w;
}

template <int D>
__global__ void __launch_bounds__(kAT, 2) attn_cc_kernel(const AttnArgs p) {
  constexpr int NP = D / 32;  // pairs of output columns a thread
  extern __shared__ __align__(16) float sm[];
  float* qt = sm;                  // [D][kAP]
  float* kt = sm + CcSmem<D>::kK;  // [D][kAP], then the weights [kAK][kAP]
  float* vs = sm + CcSmem<D>::kV;  // [kAK][D]
  __shared__ int64_t sums[kAT];
  __shared__ AttnPlan plan;
  __shared__ AttnPiece piece;
  const int tid = threadIdx.x, tx = tid & 15, ty = tid >> 4;
  attn_plan<kAK, kAT>(p, sums, &plan);
  if (tid < 2 && p.part_o != nullptr) p.part_at[2 * blockIdx.x + tid] = make_int4(kAttnWhole, 0, 0, 0);
  AttnWalk<kAK> walk;
  if (tid < 32) walk.start(p, plan, tid);
  const float* gq = static_cast<const float*>(p.q);
  const float* gk = static_cast<const float*>(p.k);
  const float* gv = static_cast<const float*>(p.v);
  const float sc = p.scale * kAttnLog2e;

  for (;;) {
    __syncthreads();
    if (tid < 32) {
      const AttnPiece w = walk.next(p);
      if (tid == 0) piece = w;
    }
    __syncthreads();
    const AttnPiece w = piece;
    if (w.tokens == 0) break;
    const int rows = w.tokens * p.group;
    // q, transposed: thread = row, chunks of 16 bytes
    for (int u = tid; u < kAR * (D / 4); u += kAT) {
      const int r = u % kAR, c = u / kAR * 4;
      float4 x = make_float4(0.f, 0.f, 0.f, 0.f);
      if (r < rows)
        x = load4(gq + (int64_t)(w.q0 + r / p.group) * p.q_stride + attn_head(p, w.kh, r % p.group) * D + c);
      put(qt + c * kAP + r, x);
    }
    int sees[4];
    float top[4], sum[4];
    float2 o[4][NP];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int r = 4 * ty + i;
      sees[i] = r < rows ? attn_sees(w, r / p.group) : 0;
      top[i] = -INFINITY;
      sum[i] = 0.f;
#pragma unroll
      for (int j = 0; j < NP; ++j) o[i][j] = make_float2(0.f, 0.f);
    }
    const bool busy = (ty & ~1) * 4 < rows;  // whether this warp has a row: a single token has a few of the 64
    const int least = attn_sees(w, 0), most = attn_sees(w, w.tokens - 1);
    for (int t = w.t0; t < w.t1; ++t) {
      const int first = t * kAK, n = most - first < kAK ? most - first : kAK;
      __syncthreads();
      // k: eight lanes along a row, which meets few lines and few banks; v: a row's lanes side by side
      for (int u = tid; u < kAK * (D / 4); u += kAT) {
        const int r = (u >> 3) % kAK, c = ((u >> 3) / kAK * 8 + (u & 7)) * 4;
        float4 x = make_float4(0.f, 0.f, 0.f, 0.f);
        if (r < n) x = load4(gk + ((int64_t)w.k0 + first + r) * p.k_stride + w.kh * D + c);
        put(kt + c * kAP + r, x);
      }
      for (int u = tid; u < kAK * (D / 4); u += kAT) {
        const int r = u / (D / 4), c = u % (D / 4) * 4;
        float4 x = make_float4(0.f, 0.f, 0.f, 0.f);
        if (r < n) x = load4(gv + ((int64_t)w.k0 + first + r) * p.v_stride + w.kh * D + c);
        *reinterpret_cast<float4*>(vs + r * D + c) = x;
      }
      __syncthreads();
      float s[4][4];
#pragma unroll
      for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int j = 0; j < 4; ++j) s[i][j] = 0.f;
      if (busy) {
#pragma unroll 8
        for (int d = 0; d < D; ++d) {
          const float4 a = *reinterpret_cast<const float4*>(qt + d * kAP + 4 * ty);
          const float4 b = *reinterpret_cast<const float4*>(kt + d * kAP + 4 * tx);
          const float av[4] = {a.x, a.y, a.z, a.w}, bv[4] = {b.x, b.y, b.z, b.w};
#pragma unroll
          for (int i = 0; i < 4; ++i)
#pragma unroll
            for (int j = 0; j < 4; ++j) s[i][j] = fmaf(av[i], bv[j], s[i][j]);
        }
      }
      __syncthreads();  // k is no longer read
      if (!busy) continue;
      const bool masked = first + kAK > least;
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        if (masked)
#pragma unroll
          for (int j = 0; j < 4; ++j)
            if (first + 4 * tx + j >= sees[i]) s[i][j] = -INFINITY;
        float m = fmaxf(fmaxf(s[i][0], s[i][1]), fmaxf(s[i][2], s[i][3]));
#pragma unroll
        for (int d = 8; d > 0; d >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, d));
        m = fmaxf(m, top[i]);
        const float base = m == -INFINITY ? 0.f : m;  // nothing seen so far: every weight is 0
        const float f = exp2f((top[i] - base) * sc);
        float l = 0.f;
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          s[i][j] = exp2f((s[i][j] - base) * sc);
          l += s[i][j];
        }
        sum[i] = fmaf(sum[i], f, l);
        top[i] = m;
#pragma unroll
        for (int j = 0; j < NP; ++j) o[i][j] = make_float2(o[i][j].x * f, o[i][j].y * f);
      }
#pragma unroll
      for (int j = 0; j < 4; ++j)
        *reinterpret_cast<float4*>(kt + (4 * tx + j) * kAP + 4 * ty) = make_float4(s[0][j], s[1][j], s[2][j], s[3][j]);
      __syncwarp();  // (a warp reads the weights of its own rows)
      if (!masked) {
#pragma unroll 4
        for (int k = 0; k < kAK; ++k) {
          const float4 a = *reinterpret_cast<const float4*>(kt + k * kAP + 4 * ty);
          const float av[4] = {a.x, a.y, a.z, a.w};
#pragma unroll
          for (int j = 0; j < NP; ++j) {
            const float2 b = *reinterpret_cast<const float2*>(vs + k * D + 32 * j + 2 * tx);
#pragma unroll
            for (int i = 0; i < 4; ++i) o[i][j] = fma2(make_float2(av[i], av[i]), b, o[i][j]);
          }
        }
      } else {
        // a key that a row does not see adds nothing to it, not even 0 times what is not finite
        for (int k = 0; k < n; ++k) {
          const float4 a = *reinterpret_cast<const float4*>(kt + k * kAP + 4 * ty);
          const float av[4] = {a.x, a.y, a.z, a.w};
#pragma unroll
          for (int j = 0; j < NP; ++j) {
            const float2 b = *reinterpret_cast<const float2*>(vs + k * D + 32 * j + 2 * tx);
#pragma unroll
            for (int i = 0; i < 4; ++i)
              if (first + k < sees[i]) o[i][j] = fma2(make_float2(av[i], av[i]), b, o[i][j]);
          }
        }
      }
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      float l = sum[i];
#pragma unroll
      for (int d = 8; d > 0; d >>= 1) l += __shfl_xor_sync(0xffffffffu, l, d);
      const int r = 4 * ty + i;
      if (r >= rows) continue;
      if (w.part != kAttnWhole) {
        const int64_t at = (int64_t)attn_slot(blockIdx.x, w.part) * p.part_rows + r;
        // The parts of a row meet by their scaled maxima, each rounded by up to
        // 2^-24 of itself. The weights here are to the one that is not: what
        // lies between them goes into the part (far off it could be anything,
        // and scores themselves are rounded by more).
        const float scaled = top[i] * sc;
        const float f = fabsf(scaled) < 65536.f ? exp2f(fmaf(top[i], sc, -scaled)) : 1.f;
#pragma unroll
        for (int j = 0; j < NP; ++j)
          *reinterpret_cast<float2*>(p.part_o + at * D + 32 * j + 2 * tx) = make_float2(o[i][j].x * f, o[i][j].y * f);
        if (tx == 0) p.part_ml[at] = make_float2(scaled, l * f);
        continue;
      }
      const int64_t token = w.q0 + r / p.group;
      const int head = attn_head(p, w.kh, r % p.group);
      float* lse = attn_lse(p, w.causal);
      float* to = attn_part_out(p, w.causal);
      if (to == nullptr) to = static_cast<float*>(p.out);
      const AttnScale f = attn_scale(top[i] * sc, l, lse != nullptr);
      to += (token * p.Hq + head) * D;
#pragma unroll
      for (int j = 0; j < NP; ++j)
        *reinterpret_cast<float2*>(to + 32 * j + 2 * tx) = make_float2(o[i][j].x * f.factor, o[i][j].y * f.factor);
      if (tx == 0 && lse != nullptr) lse[token * p.Hq + head] = f.lse;
    }
    if (tid == 0 && w.part != kAttnWhole)
      p.part_at[attn_slot(blockIdx.x, w.part)] = make_int4(w.part + 4 * w.causal, w.q0, w.tokens, w.kh);
  }
}

template <int D>
cudaError_t run(const AttnArgs& p, int grid, cudaStream_t stream) {
  constexpr int smem = CcSmem<D>::kEnd * 4;
  const cudaError_t e = cudaFuncSetAttribute(attn_cc_kernel<D>, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
  if (e != cudaSuccess) return e;
  attn_cc_kernel<D><<<grid, kAT, smem, stream>>>(p);
  return cudaGetLastError();
}
}  // namespace

int attn_cc_rows() { return kAR; }
int attn_cc_ctas(int sms) { return 2 * sms; }

cudaError_t launch_attn_cc(const AttnArgs& p, int32_t D, int grid, cudaStream_t stream) {
  switch (D) {
    case 32: return run<32>(p, grid, stream);
    case 64: return run<64>(p, grid, stream);
    case 96: return run<96>(p, grid, stream);
    default: return run<128>(p, grid, stream);
  }
}

}  // namespace gdn
