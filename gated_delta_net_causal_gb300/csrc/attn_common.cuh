// Shared device code of softmax attention over packed sequences:
//   o_t = sum_s w_ts v_s,  w_t = softmax over the visible keys s of scale q_t . k_s
// with the query heads of a key head (a "group") side by side.
//
// How the work is cut. A sequence's tokens are taken `item` at a time: an item
// is those tokens' rows (token, query head of the group) for one key head, its
// keys are read in tiles of KT. An item costs the keys that its last token
// sees, and kAttnStart tiles for its start and end; costs lie in one order
// (sequence, key head, item, key), and CTA c of G takes the c-th of G equal
// stretches of them, whatever the lengths are, cut to tiles. An item that lies
// across a border is left in parts, each (largest score, sum, unnormalised
// output) in fp32 in the workspace, and attn_join_kernel puts them together. So
// one long cache is spread over all SMs, ragged prompts leave no SM behind, and
// sums do not depend on which CTA ran first. The lengths are on the device:
// every CTA adds up the costs for itself, its threads a slice of the sequences
// each. What a CTA runs once comes from a cold instruction cache, so this is
// kept short: costs are sums of arithmetic series, where exact numbers of tiles
// would be sums of floors (3,200 to 4,000 cycles now, with the barriers and the
// TMEM set up).
#pragma once

#include "gdn_common.cuh"
#include "gdn_internal.h"

namespace gdn {

constexpr float kAttnLog2e = 1.4426950408889634f;
constexpr float kAttnLn2 = 0.69314718055994531f;

struct AttnSeq {
  int q0, qn;  // first token and number of them
  int k0, kn;  // first key row and number of them
  int causal;  // 0: a prefix, which its group's tokens see all of
};

__device__ __forceinline__ int attn_clamp(int x, int lo, int hi) { return x < lo ? lo : x > hi ? hi : x; }

// The sequences, then the groups with their prefixes.
__device__ __forceinline__ int attn_lists(const AttnArgs& p) { return p.N + p.groups; }
__device__ __forceinline__ AttnSeq attn_seq(const AttnArgs& p, int n) {
  AttnSeq s;
  s.causal = n < p.N;
  if (!s.causal) n -= p.N;
  const int32_t* cu = s.causal ? p.cu_seqlens : p.group_cu;
  const int32_t* start = s.causal ? p.kv_start : p.prefix_start;
  const int32_t* len = s.causal ? p.kv_len : p.prefix_len;
  s.q0 = attn_clamp(cu[n], 0, p.T);
  s.qn = attn_clamp(cu[n + 1], s.q0, p.T) - s.q0;
  if (start != nullptr) {
    s.k0 = attn_clamp(start[n], 0, p.kv_rows);
    s.kn = attn_clamp(len[n], 0, p.kv_rows - s.k0);
  } else {
    s.k0 = s.q0;
    s.kn = s.qn;
  }
  return s;
}

// Keys that the token at `at` of the sequence sees.
__device__ __forceinline__ int attn_visible(const AttnSeq& s, int at) {
  if (!s.causal) return s.kn;
  const int64_t v = (int64_t)s.kn - s.qn + at + 1;
  return v > 0 ? (int)v : 0;
}

// What an item costs besides its keys, in tiles. With 1, 2, 4, 6 and 8 (us):
//   bf16, one prompt of 4096 tokens, 32 / 8 heads of 128  122 110 105 108 110
//   bf16, ragged prompts of 34,482, 32 / 4 heads of 128   987 962 936 960 988
//   bf16, one prompt of 4096 tokens, 32 / 8 heads of 64    99  90  88  91  93
//   f16, chunks of 812 tokens on caches, heads of 64       94  86  80  90  90
//   bf16, 64 tokens on up to 8192 keys of 128             172 173 174 175 174
//   bf16, 64 tokens behind 8192 shared keys                60  55  61  69  77
//   f16, 52 tokens behind shared keys, heads of 96         23  22  20  20  21
//   f32, one prompt of 4096 tokens, 8 / 2 heads of 128    864 880 901 923 935
//   f32, 32 tokens on up to 8192 keys of 128              464 470 479 494 507
//   f32, 64 tokens behind 8192 shared keys                374 393 433 463 490
// So 4, which 16-bit prompts want, for all: batches behind a prefix would take
// 2, f32 (tiles of 64 keys, no start to speak of) 1.
constexpr int kAttnStart = 4;

// Keys that the last token of the item from `at` on sees.
__device__ __forceinline__ int attn_last_sees(const AttnArgs& p, const AttnSeq& s, int at) {
  return attn_visible(s, (s.qn - at < p.item ? s.qn : at + p.item) - 1);
}

// Cost of a sequence's first n items, for one key head; all but the last item
// of a sequence are full.
template <int KT>
__device__ __forceinline__ int64_t attn_cost_before(const AttnArgs& p, const AttnSeq& s, int n) {
  const int64_t start = (int64_t)n * (kAttnStart * KT);
  if (!s.causal) return start + (int64_t)n * s.kn;
  const int64_t off = (int64_t)s.kn - s.qn;  // item i's last token sees off + (i + 1) item keys
  int none = 0;                              // items that see nothing
  if (off < 0) {
    none = (int)((unsigned)-off / (unsigned)p.item);
    if (none > n) none = n;
  }
  const int64_t m = n - none;
  return start + m * off + p.item * (m * none + m * (m + 1) / 2);
}
__device__ __forceinline__ int attn_items(const AttnArgs& p, const AttnSeq& s) {
  return (int)((unsigned)(s.qn - 1) / (unsigned)p.item) + 1;
}
// Cost of a sequence for one key head.
template <int KT>
__device__ __forceinline__ int64_t attn_seq_cost(const AttnArgs& p, const AttnSeq& s) {
  if (s.qn == 0) return 0;
  return attn_cost_before<KT>(p, s, attn_items(p, s) - 1) + s.kn + kAttnStart * KT;
}

// a / b and its remainder for a >= 0, b > 0: in 32 bits where they fit, else bit by bit (the instructions of a 64-bit
// division are many, and these rarely run)
__device__ __forceinline__ int64_t attn_divide(int64_t a, int64_t b, int64_t* rest) {
  if (((a | b) >> 32) == 0) {
    const unsigned q = (unsigned)a / (unsigned)b;
    *rest = (unsigned)a - q * (unsigned)b;
    return q;
  }
  int64_t q = 0, r = 0;
#pragma unroll 1
  for (int i = 62; i >= 0; --i) {
    r = 2 * r + (a >> i & 1);
    q *= 2;
    if (r >= b) r -= b, ++q;
  }
  *rest = r;
  return q;
}

// A stretch of an item's tiles, for one CTA.
struct AttnPiece {
  int q0;     // first token of the item
  int tokens; // 0: no piece, the CTA is done
  int kh;
  int k0;     // row of the first key
  int see;    // keys that its first token sees (causal: one more for each token after it; may be negative)
  int causal; // 0: over a prefix
  int t0, t1; // tiles of this piece
  int part;   // kAttnWhole, or whether the item's tiles end with it
  int bad;    // set where a masked tile of v holds what is not finite
};
enum { kAttnWhole = 0, kAttnFirst = 1, kAttnMiddle = 2, kAttnLast = 3 };

// keys that token i of the piece sees
__device__ __forceinline__ int attn_sees(const AttnPiece& w, int i) {
  const int v = w.causal ? w.see + i : w.see;
  return v > 0 ? v : 0;
}

struct AttnPlan {
  int64_t begin, count;  // where the CTA's stretch begins, counted from sequence n, and its cost
  int n;
};

// Every thread of the CTA; sums: one of shared memory for each of them.
template <int KT, int THREADS>
__device__ __forceinline__ void attn_plan(const AttnArgs& p, int64_t* sums, AttnPlan* plan) {
  const int per = (attn_lists(p) + THREADS - 1) / THREADS;
  {
    const int64_t a = (int64_t)threadIdx.x * per, b = a + per < attn_lists(p) ? a + per : attn_lists(p);
    int64_t u = 0;
#pragma unroll 1
    for (int64_t n = a; n < b; ++n) u += attn_seq_cost<KT>(p, attn_seq(p, (int)n));
    sums[threadIdx.x] = u * p.Hk;
  }
  __syncthreads();
  if (threadIdx.x < 32) {
    constexpr int PER = THREADS / 32;
    const int lane = threadIdx.x;
    int64_t own = 0;
#pragma unroll 4
    for (int i = 0; i < PER; ++i) own += sums[lane * PER + i];
    int64_t incl = own;
#pragma unroll 1
    for (int d = 1; d < 32; d <<= 1) {
      const int64_t o = __shfl_up_sync(0xffffffffu, incl, d);
      if (lane >= d) incl += o;
    }
    const int64_t total = __shfl_sync(0xffffffffu, incl, 31);
    // no stretch is shorter than a tile, so that the parts of an item are neighbouring CTAs'
    const int64_t c = blockIdx.x, most = total / KT;
    const int64_t G = most < 1 ? 1 : most < gridDim.x ? most : gridDim.x;
    int64_t more;
    const int64_t each = attn_divide(total, G, &more);
    const int64_t u0 = each * c + (c < more ? c : more), count = c < G ? each + (c < more ? 1 : 0) : 0;
    if (lane == 0 && count == 0) *plan = AttnPlan{0, 0, 0};
    if (count > 0 && u0 >= incl - own && u0 < incl) {
      int64_t at = u0 - (incl - own);
      int i = lane * PER;
      while (at >= sums[i]) at -= sums[i++];
      *plan = AttnPlan{at, count, i * per};
    }
  }
  __syncthreads();
}

// Hands out a CTA's pieces in order. A warp's: all lanes have the same.
template <int KT>
struct AttnWalk {
  AttnSeq s;
  int64_t left, pos;  // cost left of the stretch; where in the item it goes on
  int n, kh, at;
  bool whole;  // no item is cut: those that begin in the stretch are taken to their ends

  __device__ __forceinline__ void start(const AttnArgs& p, const AttnPlan& plan, int lane) {
    left = plan.count;
    whole = p.part_o == nullptr;
    n = plan.n;
    kh = at = 0;
    pos = 0;
    if (left <= 0) return;
    // the sequence: the lanes have 32 of them
    int64_t u = plan.begin, own, incl;
    unsigned past;
    AttnSeq mine{0, 0, 0, 0, 0};
    for (;;) {
      if (n + lane < attn_lists(p)) mine = attn_seq(p, n + lane);
      else mine.qn = 0;
      own = attn_seq_cost<KT>(p, mine);
      incl = own * p.Hk;
#pragma unroll 1
      for (int d = 1; d < 32; d <<= 1) {
        const int64_t o = __shfl_up_sync(0xffffffffu, incl, d);
        if (lane >= d) incl += o;
      }
      past = __ballot_sync(0xffffffffu, incl > u);
      if (past != 0) break;
      u -= __shfl_sync(0xffffffffu, incl, 31);
      n += 32;
    }
    const int l = __ffs(past) - 1;
    n += l;
    u -= __shfl_sync(0xffffffffu, incl - own * p.Hk, l);
    s = AttnSeq{__shfl_sync(0xffffffffu, mine.q0, l), __shfl_sync(0xffffffffu, mine.qn, l),
                __shfl_sync(0xffffffffu, mine.k0, l), __shfl_sync(0xffffffffu, mine.kn, l),
                __shfl_sync(0xffffffffu, mine.causal, l)};
    kh = (int)attn_divide(u, __shfl_sync(0xffffffffu, own, l), &u);
    // the item: the last one with no more than u before it, among 32 evenly spaced ones at a time
    int lo = 0, count = attn_items(p, s);
    pos = u;
#pragma unroll 1
    while (count > 1) {
      const int step = (int)((unsigned)(count + 31) / 32);
      const int64_t rest = u - attn_cost_before<KT>(p, s, lo + lane * step);
      const int k = 31 - __clz(__ballot_sync(0xffffffffu, lane * step < count && rest >= 0));  // (lane 0's is)
      pos = __shfl_sync(0xffffffffu, rest, k);
      lo += k * step;
      count = count - k * step < step ? count - k * step : step;
    }
    at = lo * p.item;
    // the CTA before takes it to its end?
    const int seen = attn_last_sees(p, s, at);
    if (whole ? pos > 0 : (int)(pos / KT) >= (seen > KT ? (seen + KT - 1) / KT : 1)) {
      left -= seen + kAttnStart * KT - pos;
      pos = 0;
      step(p);
    }
  }
  // to the next item
  __device__ __forceinline__ void step(const AttnArgs& p) {
    if (s.qn - at > p.item) {
      at += p.item;
      return;
    }
    at = 0;
    if (++kh < p.Hk) return;
    kh = 0;
    if (left <= 0) return;  // (there may be no sequence behind the last)
    do s = attn_seq(p, ++n);
    while (s.qn == 0);
  }
  __device__ __forceinline__ AttnPiece next(const AttnArgs& p) {
    AttnPiece w{};
    if (left <= 0) return w;
    const int seen = attn_last_sees(p, s, at), keys = (seen + KT - 1) / KT, tiles = keys > 0 ? keys : 1;
    const int64_t rest = seen + kAttnStart * KT - pos;
    const int from = (int)(pos / KT);
    int to = tiles;
    if (!whole && left < rest && (pos + left) / KT < tiles) to = (int)((pos + left) / KT);
    left -= rest;
    if (to == from) return w;  // less than a tile, which the CTA after takes
    w.q0 = s.q0 + at;
    w.tokens = s.qn - at < p.item ? s.qn - at : p.item;
    w.kh = kh;
    w.k0 = s.k0;
    w.see = s.causal ? (int)((int64_t)s.kn - s.qn + at + 1) : s.kn;
    w.causal = s.causal;
    w.t0 = from < keys ? from : keys;
    w.t1 = to < keys ? to : keys;  // (no tile where one stands for none)
    w.part = from > 0 ? (to == tiles ? kAttnLast : kAttnMiddle) : (to == tiles ? kAttnWhole : kAttnFirst);
    pos = 0;
    step(p);  // (where the item goes on, so does another CTA: nothing is left here)
    return w;
  }
};

// A CTA's two places for parts: the one that its stretch begins with, and the
// one that it ends with.
__device__ __forceinline__ int attn_slot(int cta, int part) { return 2 * cta + (part == kAttnFirst ? 1 : 0); }

// query head of member m of key head kh's group
__device__ __forceinline__ int attn_head(const AttnArgs& p, int kh, int m) {
  return p.map == GDN_MAP_TILED ? m * p.Hk + kh : kh * p.group + m;
}

// Where a piece's outputs go: out, or with groups, in fp32, those over the
// sequences' keys and over the prefixes apart.
__device__ __forceinline__ float* attn_part_out(const AttnArgs& p, int causal) {
  return p.groups > 0 ? p.part_out[causal ? 0 : 1] : nullptr;
}
__device__ __forceinline__ float* attn_lse(const AttnArgs& p, int causal) {
  return p.groups > 0 ? p.part_lse[causal ? 0 : 1] : p.lse;
}

// A row's factor of its unnormalised outputs and the logarithm of its sum, from
// the largest score (times scale and log2 e) and the sum of exponentials to it.
// A row that sees nothing has a sum of 0; scores that are all NaN have no
// largest, but a sum that is NaN.
struct AttnScale {
  float factor, lse;
};
__device__ __forceinline__ AttnScale attn_scale(float top, float sum, bool lse) {
  if (sum == 0.f) return AttnScale{0.f, -INFINITY};
  return AttnScale{__frcp_rn(sum), lse ? (top + log2f(sum)) * kAttnLn2 : 0.f};
}

}  // namespace gdn
