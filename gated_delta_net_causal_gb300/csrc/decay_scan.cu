// Linear attention with a decay for each head over packed sequences, token
// by token: the state of one V head stays in the registers of a CTA while it
// goes through the tokens of a segment. Serves every type and head dim.
//
//   S = exp(g_t) S + v_t k_t^T,   o_t = scale S q_t
//
// Each lane holds NV4 * 4 columns of RPL rows (64 floats at D = 128), so a
// token costs a lane 3 paired FMAs per two elements and its q and k columns
// from shared memory; q, k, v and exp(g) of kTile tokens are staged there in
// fp32, the next tile's loads in flight in registers meanwhile, and a tile's
// outputs are normed and written one barrier later, while the next tile runs.
//
// The recurrence is a chain over the tokens, so one CTA per V head leaves
// most SMs idle for few heads and long prompts. With a workspace the tokens
// are cut into segments that run side by side: a first pass computes what
// each segment adds to the state and multiplies it by, a second one the
// outputs, each segment starting from what those before it add up to. That
// goes through the states twice; segments are as long as the SMs allow.
// Bound by the FMAs and shuffles of its few warps, and by the chain: fp32, 1024
// tokens, 32 heads 148 us (520 in one pass); 208 tokens of three sequences,
// 4 heads of 64, 9 and 11 us for the two passes.
#include <algorithm>
#include <type_traits>

#include "decay_common.cuh"

namespace gdn {
namespace {

constexpr int kTile = 8;  // tokens staged at a time

// whole: outputs, and the state after the sequence; local: the first pass
enum { kWhole = 0, kLocal = 1 };

template <typename T, int D>
struct ScanSmem {
  float q[2][kTile][D], k[2][kTile][D], v[2][kTile][D], o[2][kTile][D];
  Decay decay[2][kTile];
  int near[2];  // every token of the tile decays by less than half
};

template <typename T, int D, int MODE, bool FEW>
__global__ void __launch_bounds__(DecayGeom<D, FEW>::THREADS, FEW ? 1 : (D == 32 ? 768 : 512) / DecayGeom<D>::THREADS)
    decay_scan_kernel(const DecayArgs p, const DecaySegments sg) {
  using G = DecayGeom<D, FEW>;
  constexpr int LPR = G::LPR, NV4 = G::NV4, RPL = G::RPL, RPW = G::RPW, NT = G::THREADS;
  extern __shared__ __align__(16) unsigned char smem_raw[];
  ScanSmem<T, D>& sm = *reinterpret_cast<ScanSmem<T, D>*>(smem_raw);
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int sub = lane % LPR, rq = lane / LPR;
  const int slot = blockIdx.x / (unsigned)p.Hv;  // a segment's V heads side by side: they share q, k in L2
  const int h = blockIdx.x % (unsigned)p.Hv;
  const int kh = k_head_of(p.map, h, p.Hk, p.rep);
  DecaySegment s;
  if (!find_segment(p, sg, slot, lane, &s)) return;
  if (MODE == kLocal && s.index + 1 == s.parts) return;
  float* gS = p.state + ((int64_t)s.seq * p.Hv + h) * (int64_t)(D * D);
  float4 st[RPL][NV4];
  const DecaySlots ws(p, sg, s, h, D * D);
  const int at0 = (warp * G::WROWS + rq) * D + 4 * sub;
  if (MODE == kLocal) {
    float* keep = sg.states + ((int64_t)(s.kept + s.parts - 1) * p.Hv + h) * (D * D);
#pragma unroll
    for (int u = 0; u < RPL; ++u)
#pragma unroll
      for (int m = 0; m < NV4; ++m) {
        const int at = at0 + u * RPW * D + 4 * LPR * m;
        st[u][m] = make_float4(0.f, 0.f, 0.f, 0.f);
        if (s.index == 0) {
          st[u][m] = *reinterpret_cast<const float4*>(gS + at);
          *reinterpret_cast<float4*>(keep + at) = st[u][m];
        }
      }
  } else if (s.parts == 1) {
#pragma unroll
    for (int u = 0; u < RPL; ++u)
#pragma unroll
      for (int m = 0; m < NV4; ++m)
        st[u][m] = *reinterpret_cast<const float4*>(gS + at0 + u * RPW * D + 4 * LPR * m);
  } else {
#pragma unroll
    for (int u = 0; u < RPL; ++u) ws.start4<NV4>(s.index, s.parts, at0 + u * RPW * D, 4 * LPR, st[u]);
  }

  // staging: unit u of a tile is four elements; units of q, k, v in turn
  constexpr int UNITS = kTile * D / 4, PER = (3 * UNITS + NT - 1) / NT;
  // as they lie in memory: converting them here would wait for each load
  using Raw = typename std::conditional<sizeof(T) == 4, float4, uint2>::type;
  Raw pre[PER];
  float pre_g = 0.f;
  auto fetch = [&](int t0) {
#pragma unroll
    for (int i = 0; i < PER; ++i) {
      const int u = tid + i * NT;
      const int which = u / UNITS, r = u - which * UNITS, tt = r / (D / 4), c = (r - tt * (D / 4)) * 4;
      if (which < 3 && t0 + tt < s.end && !(MODE == kLocal && which == 0)) {
        const T* src = which == 0   ? static_cast<const T*>(p.q) + (int64_t)(t0 + tt) * p.q_stride + kh * D + c
                       : which == 1 ? static_cast<const T*>(p.k) + (int64_t)(t0 + tt) * p.k_stride + kh * D + c
                                    : static_cast<const T*>(p.v) + (int64_t)(t0 + tt) * p.v_stride + h * D + c;
        pre[i] = *reinterpret_cast<const Raw*>(src);
      }
    }
    if (tid < kTile && t0 + tid < s.end) pre_g = p.g[(int64_t)(t0 + tid) * p.g_stride + h];
  };
  float total = 0.f;  // thread tt < kTile: its share of the segment's log decay
  auto stash = [&](int buf, int t0) {
#pragma unroll
    for (int i = 0; i < PER; ++i) {
      const int u = tid + i * NT;
      const int which = u / UNITS, r = u - which * UNITS;
      if (which < 3) {
        float* dst = (which == 0 ? &sm.q[buf][0][0] : which == 1 ? &sm.k[buf][0][0] : &sm.v[buf][0][0]) + 4 * r;
        *reinterpret_cast<float4*>(dst) = load4(reinterpret_cast<const T*>(&pre[i]));
      }
    }
    if (warp == 0) {
      Decay d{0.f, 0.f};
      if (tid < kTile && t0 + tid < s.end) {
        const float g = decay_log(pre_g);
        d = decay_factor(g);
        sm.decay[buf][tid] = d;
        if (MODE == kLocal) total += g;
      }
      const bool near = __all_sync(0xffffffffu, tid >= kTile || d.keep != 0.f);
      if (tid == 0) sm.near[buf] = near;
    }
  };
  // outputs of a tile: token tt to warp tt % WARPS, each lane COLS columns; z
  // comes in while the tile runs, and a warp's tokens go side by side
  constexpr int COLS = D / 32, TOKENS = (kTile + G::WARPS - 1) / G::WARPS;
  struct alignas(COLS == 3 ? sizeof(T) : COLS * sizeof(T)) Columns {
    T v[COLS];
  };
  float nw[COLS];
#pragma unroll
  for (int e = 0; e < COLS; ++e) nw[e] = MODE == kWhole && p.z != nullptr ? p.norm_w[lane * COLS + e] : 0.f;
  Columns zr[TOKENS];
  auto fetch_z = [&](int t0) {
#pragma unroll
    for (int i = 0; i < TOKENS; ++i) {
      const int tt = warp + i * G::WARPS;
      if (p.z != nullptr && tt < kTile && t0 + tt < s.end)
        zr[i] = reinterpret_cast<const Columns*>(static_cast<const T*>(p.z) + (int64_t)(t0 + tt) * p.z_stride + h * D)[lane];
    }
  };
  auto write_tile = [&](int buf, int t0) {
    float o[TOKENS][COLS], ss[TOKENS];
#pragma unroll
    for (int i = 0; i < TOKENS; ++i) {
      const int tt = warp + i * G::WARPS;
      ss[i] = 0.f;
#pragma unroll
      for (int e = 0; e < COLS; ++e) {
        o[i][e] = tt < kTile ? sm.o[buf][tt < kTile ? tt : 0][lane * COLS + e] : 0.f;
        ss[i] += o[i][e] * o[i][e];
      }
    }
    if (p.z != nullptr) {
#pragma unroll
      for (int d = 16; d > 0; d >>= 1)
#pragma unroll
        for (int i = 0; i < TOKENS; ++i) ss[i] += __shfl_xor_sync(0xffffffffu, ss[i], d);
    }
#pragma unroll
    for (int i = 0; i < TOKENS; ++i) {
      const int tt = warp + i * G::WARPS;
      if (tt >= kTile || t0 + tt >= s.end) continue;
      const int64_t orow = ((int64_t)(t0 + tt) * p.Hv + h) * D;
      if (p.core_out != nullptr) {
#pragma unroll
        for (int e = 0; e < COLS; ++e) p.core_out[orow + lane * COLS + e] = o[i][e];
      }
      if (p.out == nullptr) continue;
      const float inv = 1.f / sqrtf(ss[i] / (float)D + p.rms_eps);
      Columns c;
#pragma unroll
      for (int e = 0; e < COLS; ++e) {
        const float y = p.z == nullptr ? o[i][e] : o[i][e] * inv * nw[e] * silu_f(to_f32(zr[i].v[e]));
        c.v[e] = from_f32<T>(y);
      }
      reinterpret_cast<Columns*>(static_cast<T*>(p.out) + orow)[lane] = c;
    }
  };

  fetch(s.begin);
  stash(0, s.begin);
  __syncthreads();
  int buf = 0;
  for (int t0 = s.begin; t0 < s.end; t0 += kTile, buf ^= 1) {
    if (t0 + kTile < s.end) fetch(t0 + kTile);
    if (MODE == kWhole) fetch_z(t0);
    const int n = s.end - t0 < kTile ? s.end - t0 : kTile;
    const auto token = [&](int tt, auto near) {
      const Decay decay = sm.decay[buf][tt];
      float4 kr[NV4];
#pragma unroll
      for (int m = 0; m < NV4; ++m) kr[m] = *reinterpret_cast<const float4*>(&sm.k[buf][tt][4 * sub + 4 * LPR * m]);
#pragma unroll
      for (int u = 0; u < RPL; ++u) {
        const float v = sm.v[buf][tt][warp * G::WROWS + u * RPW + rq];
        if constexpr (decltype(near)::value) decay_update_near<NV4>(st[u], kr, decay.factor, v);
        else decay_update<NV4>(st[u], kr, decay, v);
      }
      if (MODE == kWhole) {
        float o[RPL];
#pragma unroll
        for (int m = 0; m < NV4; ++m) kr[m] = *reinterpret_cast<const float4*>(&sm.q[buf][tt][4 * sub + 4 * LPR * m]);
#pragma unroll
        for (int u = 0; u < RPL; ++u) o[u] = row_dot<NV4>(st[u], kr);
#pragma unroll
        for (int d = LPR / 2; d > 0; d >>= 1)
#pragma unroll
          for (int u = 0; u < RPL; ++u) o[u] += __shfl_xor_sync(0xffffffffu, o[u], d);
        if (sub == 0)
#pragma unroll
          for (int u = 0; u < RPL; ++u) sm.o[buf][tt][warp * G::WROWS + u * RPW + rq] = o[u] * p.scale;
      }
    };
    // a whole tile of slow decays unrolled, so that one token's loads and sums
    // run under the next one's updates
    if (sm.near[buf]) {
#pragma unroll
      for (int tt = 0; tt < kTile; ++tt) token(tt, std::true_type());
    } else {
      for (int tt = 0; tt < n; ++tt) token(tt, std::false_type());
    }
    if (t0 + kTile < s.end) stash(buf ^ 1, t0 + kTile);
    __syncthreads();
    if (MODE == kWhole) write_tile(buf, t0);
  }

  if (MODE == kLocal || s.index + 1 == s.parts) {
    float* to = MODE == kLocal ? sg.states + ((int64_t)(s.kept + s.index) * p.Hv + h) * (D * D) : gS;
#pragma unroll
    for (int u = 0; u < RPL; ++u)
#pragma unroll
      for (int m = 0; m < NV4; ++m)
        *reinterpret_cast<float4*>(to + at0 + u * RPW * D + 4 * LPR * m) = st[u][m];
  }
  if (MODE == kLocal && warp == 0) {
    total = group_sum<32>(tid < kTile ? total : 0.f);
    if (lane == 0) sg.decays[(int64_t)(s.kept + s.index) * p.Hv + h] = expf(total);
  }
}

template <typename T, int D, bool FEW>
cudaError_t launch_scan_k(const DecayArgs& p, const DecaySegments& sg, cudaStream_t stream) {
  constexpr int smem = (int)sizeof(ScanSmem<T, D>), threads = DecayGeom<D, FEW>::THREADS;
  const unsigned grid = (unsigned)(sg.slots * p.Hv);
  if (sg.states != nullptr) {
    decay_scan_kernel<T, D, kLocal, FEW><<<grid, threads, smem, stream>>>(p, sg);
    const cudaError_t e = cudaGetLastError();
    if (e != cudaSuccess) return e;
  }
  decay_scan_kernel<T, D, kWhole, FEW><<<grid, threads, smem, stream>>>(p, sg);
  return cudaGetLastError();
}

template <typename T, int D>
cudaError_t launch_scan_td(const DecayArgs& p, const DecaySegments& sg, cudaStream_t stream) {
  return sg.slots * p.Hv <= 152 ? launch_scan_k<T, D, true>(p, sg, stream) : launch_scan_k<T, D, false>(p, sg, stream);
}

template <typename T>
cudaError_t launch_scan_t(const DecayArgs& p, const DecaySegments& sg, int32_t D, cudaStream_t stream) {
  switch (D) {
    case 32: return launch_scan_td<T, 32>(p, sg, stream);
    case 64: return launch_scan_td<T, 64>(p, sg, stream);
    case 96: return launch_scan_td<T, 96>(p, sg, stream);
    case 128: return launch_scan_td<T, 128>(p, sg, stream);
    default: return cudaErrorInvalidValue;
  }
}

}  // namespace

// Sized for the 152 SMs of the one target, so that a workspace asked for on
// one thread fits the call on another: as many segments as give every SM one
// CTA (token by token: two) and no CTA a second turn, as many to a sequence if
// they are alike, else (and token by token, but for a lone sequence) with room
// for a half full last one of each. With few heads that would be many short
// ones, and the last of them reads the states that all others add: on the
// tensor cores a chunk of 64 tokens costs about as much as seven such states,
// so n chunks in segments of m cost m + n / (7 m), least at m = sqrt(n / 7);
// token by token a state costs about as much as two tokens (whatever D: both
// go with the state's size), so n tokens in segments of m cost 2 m + 2 n / m,
// least at m = sqrt(n).
// On the tensor cores n chunks take 8 + 2.65 n us in one pass and 17 + 4.2 m +
// 0.5 n / m in two over segments of m, so short prompts and those of many
// heads stay whole (one prompt, 32 heads, one pass and two: 128 tokens 13 and
// 20 us, 512 tokens 29 and 26, 2048 tokens 93 and 50). Where that holds for
// sequences of the mean length, one of three times that may still gain: those
// above the mean by a quarter are cut alone. (Measured with one bf16 part of S
// and P in the output pass. With the two that it has a chunk takes 0.35 us
// more, 7 + 3.0 n and 17 + 4.4 m + 0.5 n / m, which would move the border by
// less than a chunk: 512 tokens 31 us in one pass and 27 as cut, 4096 200 and
// 89.)
// Token by token many (sequence, V head) pairs hide long ones among them, whose
// chain of tokens outlasts the rest: sequences of half more tokens than an even
// share of the SMs' work are then cut, too (fp32, 64 heads, 13 sequences of
// 9782 tokens in all, the longest 3660: 1574 us and uncut 2251 at head_dim 64,
// 2501 and 2805 at 128; 20 of 1000 tokens, which nothing cuts, 1484 and 1466,
// for the first pass that finds nothing to do).
void decay_cut(int32_t N, int64_t T, int32_t Hv, int32_t D, bool chunks, DecaySegments* sg) {
  sg->len = sg->whole = (int32_t)T + 1;
  if (T == 0) return;
  if (chunks) {
    const int64_t n = (T + 63) / 64, sms = 152 / Hv, each = sms / N;
    const int64_t more = each >= 2 ? N * each : sms - N / 2;
    if (more < 1) return;
    int64_t len = (n + more - 1) / more;
    while (7 * N * len * len < n) ++len;
    if (each >= 2 && 53 * n > (84 * len + 180) * N + 10 * n / len) {
      sg->len = sg->whole = (int32_t)(64 * len);
    } else if (53 * std::min(N * n, 3 * n) > (31 * len + 180) * N + 53 * n + 10 * n / len) {
      sg->len = (int32_t)(64 * len);
      sg->whole = (int32_t)std::min<int64_t>(64 * std::max(len, (5 * n + 4 * N - 1) / (4 * N)), T);
    }
    return;
  }
  const int64_t more = N == 1 ? 304 / Hv : (608 / Hv - N) / 2, share = T * Hv / 304;
  const bool few = more >= (N == 1 || D > 64 ? 1 : 4);
  if (T <= 32 || (!few && (T <= 512 || N * (int64_t)Hv > 8192))) return;
  int64_t len = few ? (T + more - 1) / more : share / 2;
  len = (len + kTile - 1) / kTile * kTile;  // below T + kTile
  const int64_t n = (T + kTile - 1) / kTile;
  while (8 * (len / kTile) * (len / kTile) < n) len += kTile;  // 8 tokens a tile: m^2 >= T
  const int64_t whole = few ? len : std::max(len, share + share / 2);
  if (whole >= T) return;
  sg->len = (int32_t)len;
  sg->whole = (int32_t)whole;
}

cudaError_t launch_decay_scan(const DecayArgs& p, const DecaySegments& sg, int32_t dtype, int32_t D,
                              cudaStream_t stream) {
  switch (dtype) {
    case GDN_F16: return launch_scan_t<__half>(p, sg, D, stream);
    case GDN_BF16: return launch_scan_t<__nv_bfloat16>(p, sg, D, stream);
    case GDN_F32: return launch_scan_t<float>(p, sg, D, stream);
    default: return cudaErrorInvalidValue;
  }
}

}  // namespace gdn

GDN_DEFINE_ERROR_READER(decay_scan)
