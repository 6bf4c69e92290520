// Device side of rcp_score_mod: which cached tokens a query row sees, and what happens to its
// scores before the softmax.  Shared by the decode and prefill kernels.
#pragma once
#include <cstdint>

#include "ptx.cuh"
#include "shape.h"

namespace rcp {

// What a row at position pos of a request with L tokens sees: tokens t < pfx, and tokens
// lo <= t <= pos (lo >= pos + 1: none of those).
struct RowView {
  int32_t pfx, lo;
};

__device__ __forceinline__ int32_t view_prefix(const AttnParams& p, int b, int32_t L) {
  const int32_t f = p.prefix_lens ? p.prefix_lens[b] : 0;
  return f < 0 ? 0 : (f < L ? f : L);
}
// First token behind the prefix that row `row` (of the call's query rows), at position pos,
// may see: the later of its row_begin and its window's start.
__device__ __forceinline__ int32_t view_begin(const AttnParams& p, int64_t row, int32_t pos) {
  int32_t lo = p.row_begin ? p.row_begin[row] : 0;
  if (p.window > 0 && pos + 1 - p.window > lo) lo = pos + 1 - p.window;
  return lo > 0 ? lo : 0;
}

// The position a row's distance bias is measured from: its own when it sees itself, else the
// last token of the prefix.  The softmax does not change when a constant is added to a row's
// scores, so only differences of distances count; measured from the nearest visible token
// the bias of the tokens that carry weight stays small, and fp32 exact to its last bits.
__device__ __forceinline__ int32_t bias_origin(RowView v, int32_t pos) {
  return (v.lo <= pos || pos < v.pfx) ? pos : v.pfx - 1;
}
// Distance of the farthest token that the row sees from that position: what a bias that grows
// with the distance is measured from in its turn (the prefill).
__device__ __forceinline__ int32_t bias_reach(RowView v, int32_t pos, int32_t org) {
  const int32_t first = v.pfx > 0 ? 0 : v.lo;
  const int32_t last = v.lo <= pos && pos >= v.pfx ? pos : v.pfx - 1;
  const int32_t a = org - first, b = last - org;
  return a > b ? a : b;
}

// A prefill request's key tiles (KT keys) that some of its rows sees: those of the prefix and
// those from the least first token of any row on, from the plan's (prefix, least first token).
// Their pages, one after another, are the rows of V^ (reconstructing variant) and the pages
// the widening pass copies; key tile x is number x among them, or x - (lt - np) past the prefix.
template <class S>
struct TileMap {
  static constexpr int KT = PrefillCfg<S>::KT, BPT = KT / kBlockSize;
  int32_t pfx, lo, np, lt, nblk;   // np prefix tiles, then tiles lt .. ; pages of the request
  __device__ __forceinline__ TileMap(const int32_t* m, int32_t nb) : pfx(m[0]), lo(m[1]), nblk(nb) {
    const int32_t tiles = (nblk + BPT - 1) / BPT;
    np = (pfx + KT - 1) / KT;
    lt = lo / KT;
    if (lo >= nblk * kBlockSize || lt > tiles) lt = tiles;
    if (lt < np) lt = np;
  }
  __device__ __forceinline__ int32_t pages() const {
    const int32_t a = np * BPT < nblk ? np * BPT : nblk, b = nblk - lt * BPT;
    return a + (b > 0 ? b : 0);
  }
  // page of the request that is number j of them
  __device__ __forceinline__ int32_t page(int32_t j) const {
    return j < np * BPT ? j : (lt - np) * BPT + j;
  }
  // whether some row may see a token of page x (another one's table entry is not looked at)
  __device__ __forceinline__ bool seen(int32_t x) const {
    return x * kBlockSize < pfx || (x + 1) * kBlockSize > lo;
  }
};

// cap2 tanh(x / cap2) of a pair of scores, log2 units, for the prefill, where a row meets 128
// of them per tile and the FMA pipe sets the pace: six operations per score.  Scores up to 0.7
// of the cap take a polynomial: with u = x / cap2 and v = u^2, tanh(u) / u = 1 + v q(v), q a fit
// of degree 3 on v in [0, 0.49] (relative error 3.8e-7, in fp32 arithmetic 4.5e-7; absolute
// 2.7e-7 of the cap).  CapNear holds its coefficients in powers of x^2, c_k / cap2^(2k), within fp32 for
// every cap allowed.  wmax collects the largest x^2; the caller takes cap_far if it passed
// w_near = (0.7 cap2)^2.
struct CapNear {
  float c1, c2, c3, c4, w_near;
  __device__ __forceinline__ explicit CapNear(float cap2, float inv_cap2) {
    const float i2 = inv_cap2 * inv_cap2;
    c1 = -0.333311808f * i2;
    c2 = 0.132888389f * i2 * i2;
    c3 = -0.0510577062f * i2 * i2 * i2;
    c4 = 0.013981962f * i2 * i2 * i2 * i2;
    w_near = 0.49f * cap2 * cap2;
  }
};
__device__ __forceinline__ float2 both(float x) { return make_float2(x, x); }
__device__ __forceinline__ float2 cap_pair_near(float2 x, const CapNear& k, float& wmax) {
  const float2 w = mul_f32x2(x, x);
  float2 q = fma_f32x2(both(k.c4), w, both(k.c3));
  q = fma_f32x2(q, w, both(k.c2));
  q = fma_f32x2(q, w, both(k.c1));
  wmax = max3f(wmax, w.x, w.y);
  return fma_f32x2(mul_f32x2(x, w), q, x);
}
// Any score: 1 - 2 / (e^2u + 1), absolute error about 3e-7 of the cap as well (the two
// approximate instructions' 2^-22 and 2^-23): at the largest cap allowed, 1024, 3e-4 of a unit,
// less than the rounding of its weights to fp16.  The decode, which has few scores per lane and
// page, takes it for all (a call of tanhf cost 17 % of the E4M3 step at 64 x 8192).
__device__ __forceinline__ float cap_score(float x, float cap2, float inv_cap2) {
  const float e = fast_exp2(x * (2.88539008f * inv_cap2));
  return fmaf(-2.f * cap2, fast_rcp(e + 1.f), cap2);
}
__device__ __forceinline__ float2 cap_pair_far(float2 x, float cap2, float twice_inv) {
  const float2 a = mul_f32x2(x, both(twice_inv));   // twice_inv = 2 log2(e) / cap2
  const float2 e = add_f32x2(make_float2(fast_exp2(a.x), fast_exp2(a.y)), both(1.f));
  return fma_f32x2(make_float2(fast_rcp(e.x), fast_rcp(e.y)), both(-2.f * cap2), both(cap2));
}

// Bits c of a 32-column word starting at column c0 whose columns lie in [a, b).
__device__ __forceinline__ uint32_t column_bits(int32_t a, int32_t b, int32_t c0) {
  const int32_t lo = a - c0, hi = b - c0;
  const uint32_t up = hi >= 32 ? 0xFFFFFFFFu : hi <= 0 ? 0u : (1u << hi) - 1u;
  const uint32_t dn = lo >= 32 ? 0xFFFFFFFFu : lo <= 0 ? 0u : (1u << lo) - 1u;
  return up & ~dn;
}

// A prefill row's modifications: what it sees, where its bias starts from (log2 units per
// token; reach: the distance at which it is zero), and whether one of its warp's scores has passed the range of the cap's polynomial.
struct RowMod {
  RowView view;
  int32_t pos, org;
  float slope2, reach;
  bool far;
  CapNear near;
  __device__ __forceinline__ RowMod(const AttnParams& p, int head, bool row_ok, int64_t row,
                                    int32_t pos_, int32_t pfx)
      : view{pfx, row_ok ? view_begin(p, row, pos_) : 0}, pos(pos_), org(bias_origin(view, pos_)),
        slope2(p.slopes ? p.slopes[head] * 1.44269504f : 0.f),
        reach(slope2 < 0.f ? static_cast<float>(bias_reach(view, pos, org)) : 0.f), far(false),
        near(p.cap2, p.inv_cap2) {
    if (!row_ok) near.w_near = INFINITY;   // a row outside the chunk has no say in the form
  }
  // the 32 keys from t0 on that the row sees, without the rejected pages (two bits of bad)
  __device__ __forceinline__ uint32_t seen(int32_t t0, uint32_t bad) const {
    uint32_t w = column_bits(0, view.pfx, t0) | column_bits(view.lo, pos + 1, t0);
    if (bad & 1u) w &= 0xFFFF0000u;
    if (bad & 2u) w &= 0x0000FFFFu;
    return w;
  }
};

// Cap and bias of a row's scores of the keys h0 .. h0 + KC - 1, and -inf for those it does not
// see (edge: seen[] says which; else it sees them all).  reload() reads the scores again.
// Returns what has to be added to every score.
template <int KC, class Reload>
__device__ __forceinline__ float modify_scores(float (&sv)[KC], const AttnParams& p, RowMod& rm,
                                               int32_t h0, bool edge,
                                               const uint32_t (&seen)[KC / 32], Reload reload) {
  float shift = 0.f;
  if (p.cap2 > 0.f) {
    if (!rm.far) {
      // which form the cap takes must not depend on what hidden slots hold
      if (edge) {
#pragma unroll
        for (int c = 0; c < KC; ++c) sv[c] = (seen[c / 32] >> (c % 32)) & 1u ? sv[c] : 0.f;
      }
      float wmax = 0.f;
#pragma unroll
      for (int c = 0; c < KC; c += 2) {
        const float2 y = cap_pair_near(make_float2(sv[c], sv[c + 1]), rm.near, wmax);
        sv[c] = y.x;
        sv[c + 1] = y.y;
      }
      if (__any_sync(0xffffffffu, !(wmax <= rm.near.w_near))) {
        // some score is past the polynomial's range; the warp stays with the general form
        rm.far = true;
        reload();
      }
    }
    if (rm.far) {
      const float twice_inv = 2.88539008f * p.inv_cap2;
#pragma unroll
      for (int c = 0; c < KC; c += 2) {
        const float2 y = cap_pair_far(make_float2(sv[c], sv[c + 1]), p.cap2, twice_inv);
        sv[c] = y.x;
        sv[c + 1] = y.y;
      }
    }
  }
  if (p.slopes) {
    // Every key at or before the origin: slope (t - org), the part they share kept apart.  The
    // row's maximum then holds that part, and the weights are off by up to its rounding (2^-4
    // below 2^20; past it they could leave fp16's range).  A bias that grows with the distance
    // is largest where that part is: no key is worked out so.
    const float part = rm.slope2 * static_cast<float>(h0 - rm.org);
    if (__all_sync(0xffffffffu, h0 + KC - 1 <= rm.org && part <= 0.f && part > -1048576.f)) {
      shift = part;
#pragma unroll
      for (int c = 0; c < KC; ++c) sv[c] = fmaf(rm.slope2, static_cast<float>(c), sv[c]);
    } else {
      const float d0 = static_cast<float>(rm.org - h0);
#pragma unroll
      for (int c = 0; c < KC; ++c)
        sv[c] = fmaf(-rm.slope2, fabsf(d0 - static_cast<float>(c)) - rm.reach, sv[c]);
    }
  }
  if (edge) {
#pragma unroll
    for (int c = 0; c < KC; ++c) sv[c] = (seen[c / 32] >> (c % 32)) & 1u ? sv[c] : -INFINITY;
  }
  return shift;
}

}  // namespace rcp
