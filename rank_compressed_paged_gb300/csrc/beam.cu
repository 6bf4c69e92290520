// Beam search's selection: the best continuations of every request over its beams and the
// vocabulary, from the logits as the model left them.
//
//     total(i, t) = scores[i] + x[i][t] - M_i - log sum_u exp(x[i][u] - M_i),  M_i = max_u x[i][u]
//
// Two launches.  The scan reads the logits once: a CTA takes a segment of one row, a warp a part
// of it in sub-blocks of four words of 16 bytes per lane, the next one on its way.  It leaves the
// segment's largest logit, its sum of exponentials and its best K logits in order: within a
// row totals are ordered as logits, so no other candidate can be kept, whatever the row's sum
// turns out to be.  The merge, a CTA per request, joins the sums, works out the totals of the
// segments' candidates and takes the best K.
//
// The best K of a segment without sorting it: of each warp the T-th largest of its lanes' maxima is
// taken, T = ceil(K / 4), and of the eight warps' the ceil(K / T)-th largest.  At least K logits reach
// that bound and, unless they sit together, few more (about 15 of 131072 for K = 8).  The lanes'
// sub-blocks whose maximum reaches it are read again, from L2, their words shared out over the warp,
// and what does is listed and ranked by counting.  Where more than kListMax do (a row of equal
// logits, a sorted one), each warp finds the best K of its own part, bisecting the K-th largest where
// even they are too many.
//
// Accuracy: within a row candidates are in the order of their logits, exactly.  Candidates of different
// beams may lie within an fp32 rounding of each other, so totals are compared as sums of two fp32
// values (TwoFloat, 48 bits), in which x - M is exact.  What is left is the sum of exponentials: its
// logarithm is within 3.6e-6 if every error had the same sign (a term is off by ex2's 2^-22, by the
// rounding of its argument, 2^-20 of a unit at the most, and by 1.4e-8 of it, what fp32 drops of
// log2 e; about 32 additions on a term's way round by 2^-24 each), and was within 3e-7 on random
// rows, 5e-7 on rows of equal logits.  Beams whose totals are nearer than that may come in either order.
//
// Words are a row's own (8 or 4 tokens from its start), and a lane's terms, and the order in which
// they and the lanes' sums are added, go by the token alone.  So beams with the same logits have the
// same sum, bit for bit, and totals that are equal keep the order of (i, t).  Where the vocabulary is no
// multiple of 8 (4) a row starts inside a 16-byte word, and its words are put together from two, a
// neighbouring lane's among them.
//
// The logits are read once, everything else is a few KB per request: 64 x 8 x 131071 bf16 is 134 MB,
// 20 us at the copy rate, and takes 34.5, of 131072 tokens 32: putting the words together costs 2.2 in
// issue slots (fp16 3.6, fp32 0.6).  With shifts that are constants, in a branch for each of the seven
// starts, it cost 1.2 more, with a copy of the loop for each 7 to 16: rows that start differently then
// take turns in an SM's instruction cache.  Of the 32 the stream alone, without exponentials, takes about 24, 2.5 from there to the lists, 5 the
// merge.  All CTAs are resident at once and end together, so what follows the stream is paid in full:
// with a bound, a list and a ranking of its own for every warp the call took 4 more, with parts of
// 2048 words 5, with a segment in registers and bisected there 15.  Four CTAs per SM; five or six,
// with fewer registers, were slower (by 10).  One request of 4 x 32768 takes 7.0 us, two launches of
// little work, with parts halved until the SMs have a CTA each.
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include <cfloat>
#include <cstdint>

#include "launch.h"
#include "ptx.cuh"
#include "rcp.h"
#include "shape.h"

namespace rcp {

constexpr int kScanThreads = kBeamScanThreads, kScanWarps = kScanThreads / 32;
constexpr int kNoteMax = 128;        // sub-blocks of a lane that are read again at a time
constexpr int kListMax = 128;        // a warp's candidates that are ranked by counting
constexpr int kMergeThreads = 256;

// A total order of fp32 values as unsigned integers; 0 is below every number.
__device__ __forceinline__ uint32_t order32(float x) {
  const uint32_t b = __float_as_uint(x);
  return b ^ (b >> 31 ? 0xFFFFFFFFu : 0x80000000u);
}
__device__ __forceinline__ float value32(uint32_t o) {
  return __uint_as_float(o ^ (o >> 31 ? 0x80000000u : 0xFFFFFFFFu));
}
// Order of a row's candidates: larger logits first (-0 and +0 are equal), then lower indexes.
__device__ __forceinline__ uint64_t list_key(float x, int t) {
  return static_cast<uint64_t>(order32(x + 0.f)) << 32 | ~static_cast<uint32_t>(t);
}

// Logits of a 16-byte word.  most: their largest, NaN if one is; clean: NaN to -inf, +inf to the
// type's largest value, so that a row's maximum is finite and differences from it are no NaN.
template <class T>
struct Logits;

template <>
struct Logits<float> {
  static constexpr int VEC = 4;
  static constexpr uint32_t kHidden = 0xFF800000u;   // -inf
  static __device__ __forceinline__ float one(float x) { return fminf(fmaxf(x, -INFINITY), FLT_MAX); }
  static __device__ __forceinline__ uint32_t clean(uint32_t w) { return __float_as_uint(one(__uint_as_float(w))); }
  struct Most {
    float m = -INFINITY;
    __device__ __forceinline__ void add(uint4 w) {
      asm("max.NaN.f32 %0, %0, %1, %2;" : "+f"(m) : "f"(__uint_as_float(w.x)), "f"(__uint_as_float(w.y)));
      asm("max.NaN.f32 %0, %0, %1, %2;" : "+f"(m) : "f"(__uint_as_float(w.z)), "f"(__uint_as_float(w.w)));
    }
    __device__ __forceinline__ float value() const { return m; }
  };
  static __device__ __forceinline__ void unpack(uint4 w, float (&x)[VEC]) {
    x[0] = __uint_as_float(w.x); x[1] = __uint_as_float(w.y);
    x[2] = __uint_as_float(w.z); x[3] = __uint_as_float(w.w);
  }
  static __device__ __forceinline__ uint32_t bits(float x) { return __float_as_uint(x); }
};

template <class T, class T2>
struct Logits16 {
  static constexpr int VEC = 8;
  static __device__ __forceinline__ T2 pair(uint32_t w) { return *reinterpret_cast<const T2*>(&w); }
  static __device__ __forceinline__ uint32_t word(T2 p) { return *reinterpret_cast<const uint32_t*>(&p); }
  static __device__ __forceinline__ uint32_t bits(T x) { return *reinterpret_cast<const uint16_t*>(&x); }
};

template <>
struct Logits<__half> : Logits16<__half, __half2> {
  static constexpr uint32_t kHidden = 0xFC00FC00u;
  static __device__ __forceinline__ uint32_t clean(uint32_t w) {
    return word(__hmin2(__hmax2(pair(w), pair(kHidden)), pair(0x7BFF7BFFu)));
  }
  static __device__ __forceinline__ float one(__half x) {
    return fminf(fmaxf(__half2float(x), -INFINITY), 65504.f);
  }
  struct Most {
    __half2 m = pair(kHidden);
    __device__ __forceinline__ void add(uint4 w) {
      m = __hmax2_nan(m, __hmax2_nan(__hmax2_nan(pair(w.x), pair(w.y)), __hmax2_nan(pair(w.z), pair(w.w))));
    }
    __device__ __forceinline__ float value() const {
      return __half2float(__hmax_nan(__low2half(m), __high2half(m)));
    }
  };
  static __device__ __forceinline__ void unpack(uint4 w, float (&x)[VEC]) {
    const uint32_t v[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      const float2 f = __half22float2(pair(v[k]));
      x[2 * k] = f.x; x[2 * k + 1] = f.y;
    }
  }
};

template <>
struct Logits<__nv_bfloat16> : Logits16<__nv_bfloat16, __nv_bfloat162> {
  static constexpr uint32_t kHidden = 0xFF80FF80u;
  static __device__ __forceinline__ uint32_t clean(uint32_t w) {
    return word(__hmin2(__hmax2(pair(w), pair(kHidden)), pair(0x7F7F7F7Fu)));
  }
  static __device__ __forceinline__ float one(__nv_bfloat16 x) {
    return fminf(fmaxf(__bfloat162float(x), -INFINITY), __uint_as_float(0x7F7F0000u));
  }
  struct Most {
    __nv_bfloat162 m = pair(kHidden);
    __device__ __forceinline__ void add(uint4 w) {
      m = __hmax2_nan(m, __hmax2_nan(__hmax2_nan(pair(w.x), pair(w.y)), __hmax2_nan(pair(w.z), pair(w.w))));
    }
    __device__ __forceinline__ float value() const {
      return __bfloat162float(__hmax_nan(__low2bfloat16(m), __high2bfloat16(m)));
    }
  };
  static __device__ __forceinline__ void unpack(uint4 w, float (&x)[VEC]) {
    const uint32_t v[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
    for (int k = 0; k < 4; ++k) {   // the 16 bits are the upper half of the fp32 value
      x[2 * k] = __uint_as_float(v[k] << 16);
      x[2 * k + 1] = __uint_as_float(v[k] & 0xFFFF0000u);
    }
  }
};

// A row's words from 16-byte words, SKIP registers and `shift` bits into which they start.  w: this
// lane's of a sub-block (word k: 32 k + lane), in which the row's words end; they start in the words
// before, which lane - 1 has, or for lane 0 lane 31, one k earlier (carry: of the sub-block before; left
// for the next).
template <int SKIP>
__device__ __forceinline__ void align_words(uint4 (&w)[4], uint4& carry, int lane, int shift) {
  const uint4 last = w[3];
#pragma unroll
  for (int k = 3; k >= 0; --k) {
    const uint4 p = k ? w[k ? k - 1 : 0] : carry;
    const uint32_t own[4] = {w[k].x, w[k].y, w[k].z, w[k].w}, before[4] = {p.x, p.y, p.z, p.w};
    uint32_t c[8];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      c[i] = i < SKIP ? 0u : __shfl_sync(0xffffffffu, lane == 31 ? before[i] : own[i], (lane + 31) & 31);
      c[4 + i] = own[i];
    }
    w[k] = make_uint4(__funnelshift_r(c[SKIP], c[SKIP + 1], shift), __funnelshift_r(c[SKIP + 1], c[SKIP + 2], shift),
                      __funnelshift_r(c[SKIP + 2], c[SKIP + 3], shift),
                      __funnelshift_r(c[SKIP + 3], c[SKIP + 4], shift));
  }
  carry = last;
}

template <class T>
struct ScanSmem {
  T most[kScanWarps][beam_part_words(sizeof(T)) / 128][32];   // every lane's largest of each sub-block
  uint64_t list[kScanWarps][kListMax];       // (list_key) what reaches the bound; of a warp's part
  uint64_t best[kScanWarps * 32];            // the warps' best, K each
  float2 stat[kScanWarps];                   // the warps' largest logit and sum
  uint32_t high[kScanWarps];                 // the warps' T-th largest lane maximum (order32)
  uint32_t count[kScanWarps], reached;       // how many a list would hold
  uint16_t note[kScanWarps][kNoteMax];       // (sub-block, lane) to be read again
};

template <class T>
__global__ void __launch_bounds__(kScanThreads, 4) beam_scan_kernel(const BeamParams p) {
  using G = Logits<T>;
  constexpr int VEC = G::VEC;
  __shared__ ScanSmem<T> sm;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const uint32_t K = static_cast<uint32_t>(p.beams);
  const int row = blockIdx.x / p.splits, split = blockIdx.x - row * p.splits;
  // The row's words: word g holds tokens g VEC .. g VEC + VEC - 1, wherever the row starts, so that rows
  // with the same logits are summed and listed alike and totals that are equal stay equal.  In memory
  // word g starts `lead` logits into 16-byte word g (from src) and, if lead is not 0, ends in the next.
  // This warp: words a0 .. a1 - 1
  const int64_t r0 = static_cast<int64_t>(row) * p.vocab, w0 = r0 / VEC;
  const int lead = static_cast<int>(r0 - w0 * VEC), next = lead > 0 ? 1 : 0;
  const int words = (p.vocab + VEC - 1) / VEC;
  const int a0 = split * p.seg_words + warp * p.part_words;
  const int a1 = min(words, min((split + 1) * p.seg_words, a0 + p.part_words));
  const int subs = a1 > a0 ? (a1 - a0 + 127) / 128 : 0;
  const uint4* src = static_cast<const uint4*>(p.logits) + w0;
  // the buffer may end inside a 16-byte word: `whole` are there in full, and with them the tokens below
  // `safe`
  const int whole = static_cast<int>(
      min(static_cast<int64_t>(words) + 1, static_cast<int64_t>(p.batch) * p.beams * p.vocab / VEC - w0));
  const int safe = whole * VEC - lead;
  // words with odd logits: from odd1 on (past the vocabulary, or not in a whole 16-byte word), and the
  // one that ends a sequence, which is the merge's
  const int odd1 = min(p.vocab / VEC, max(safe, 0) / VEC);
  const int odd2 = p.eos >= 0 ? p.eos / VEC : -1;
  const uint4 hidden = make_uint4(G::kHidden, G::kHidden, G::kHidden, G::kHidden);
  // the 16-byte word in which word g ends
  auto load = [&](int g) { return g < a1 && g + next < whole ? src[g + next] : hidden; };
  // hides a word's odd logits, and loads those of an open 16-byte word
  auto mend = [&](int g, uint4& w) {
    if (g >= a1 || (g < odd1 && g != odd2)) return;
    uint32_t v[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
    for (int e = 0; e < VEC; ++e) {
      const int t = g * VEC + e;
      const uint32_t mask = VEC == 4 ? 0xFFFFFFFFu : 0xFFFFu << ((e & 1) * 16);
      uint32_t& x = v[e * 4 / VEC];
      if (t >= p.vocab || t == p.eos)
        x = (x & ~mask) | (G::kHidden & mask);
      else if (t >= safe)
        x = (x & ~mask) | G::bits(static_cast<const T*>(p.logits)[r0 + t]) << (VEC == 4 ? 0 : (e & 1) * 16);
    }
    w = make_uint4(v[0], v[1], v[2], v[3]);
  };
  auto largest = [&](const uint4 (&w)[4]) {
    typename G::Most m;
#pragma unroll
    for (int k = 0; k < 4; ++k) m.add(w[k]);
    return m.value();
  };
  auto clean = [&](uint4 (&w)[4]) {
#pragma unroll
    for (int k = 0; k < 4; ++k)
      w[k] = make_uint4(G::clean(w[k].x), G::clean(w[k].y), G::clean(w[k].z), G::clean(w[k].w));
  };
  if (lane == 0) sm.count[warp] = 0;
  if (tid == 0) sm.reached = 0;
  griddep_wait();                  // the logits are written
  griddep_launch();
  // ---- this lane's largest logit m and its sum s of exp(x - m)
  float m = -INFINITY, s = 0.f;
  uint4 w[4], ahead[4], carry = hidden;   // carry: (lane 31) the 16-byte word before a sub-block's
  constexpr int kBytes = sizeof(T);
  const int skip = lead * kBytes / 4, shift = lead * kBytes % 4 * 8;
  auto load_sub = [&](int first) {
    if (first + 128 <= min(a1, whole - next)) {
      const uint4* at = src + next + first + lane;
#pragma unroll
      for (int k = 0; k < 4; ++k) ahead[k] = at[32 * k];
    } else {
#pragma unroll
      for (int k = 0; k < 4; ++k) ahead[k] = load(first + 32 * k + lane);
    }
  };
  load_sub(a0);
  if (next && subs > 0 && a0 < whole) carry = src[a0];
#pragma unroll 1
  for (int sub = 0; sub < subs; ++sub) {
    const uint32_t first = a0 + sub * 128;
#pragma unroll
    for (int k = 0; k < 4; ++k) w[k] = ahead[k];
    if (sub + 1 < subs) load_sub(first + 128);
    if (next) {
      if (skip == 0) align_words<0>(w, carry, lane, shift);
      else if (skip == 1) align_words<1>(w, carry, lane, shift);
      else if (skip == 2) align_words<2>(w, carry, lane, shift);
      else align_words<3>(w, carry, lane, shift);
      if (first + 128 > static_cast<uint32_t>(a1)) {   // (the next part's)
#pragma unroll
        for (int k = 0; k < 4; ++k)
          if (first + 32 * k + lane >= static_cast<uint32_t>(a1)) w[k] = hidden;
      }
    }
    if (first + 128 > static_cast<uint32_t>(odd1) || odd2 - first < 128u) {
#pragma unroll
      for (int k = 0; k < 4; ++k) mend(first + 32 * k + lane, w[k]);
    }
    float mx = largest(w);
    if (!(mx < INFINITY)) {        // a NaN or +inf among them
      clean(w);
      mx = largest(w);
    }
    sm.most[warp][sub][lane] = T(mx);   // (one of them: exact)
    if (mx > m) {
      s *= fast_exp2((m - mx) * 1.44269502f);
      m = mx;
    }
    if (fabsf(m) <= 8.5e37f) {
      // exp(x - m) = 2^(x log2 e + c): one fma with c = -m log2 e rounded, whose rounding, the
      // same for every term, is undone in the sub-block's sum
      constexpr float kLog2e = 1.44269502f;
      const float c = -(m * kLog2e), off = fmaf(m, kLog2e, c);   // off: what c lacks
      float2 acc[2] = {make_float2(0.f, 0.f), make_float2(0.f, 0.f)};
      const float2 k2 = make_float2(kLog2e, kLog2e), c2 = make_float2(c, c);
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        if (first + 32 * k >= static_cast<uint32_t>(a1)) break;   // (the part's last sub-block)
        float x[VEC];
        G::unpack(w[k], x);
#pragma unroll
        for (int e = 0; e < VEC; e += 2) {
          const float2 a = fma_f32x2(make_float2(x[e], x[e + 1]), k2, c2);
          acc[(e >> 1) & 1] =
              add_f32x2(acc[(e >> 1) & 1], make_float2(fast_exp2(a.x), fast_exp2(a.y)));
        }
      }
      const float2 t = add_f32x2(acc[0], acc[1]);
      const float part = t.x + t.y;
      s += fmaf(part, -0.693147182f * off, part);
    } else if (m > -INFINITY) {    // past 2^126 that product may leave fp32's range
#pragma unroll 1
      for (int k = 0; k < 4; ++k) {
        const uint4 wk = k == 0 ? w[0] : k == 1 ? w[1] : k == 2 ? w[2] : w[3];
        float x[VEC];
        G::unpack(wk, x);
#pragma unroll 1
        for (int e = 0; e < VEC; ++e) s += expf(x[e] - m);
      }
    }
  }
  // ---- the warp's largest, its sum, and the K-th largest of its lanes
  float M = m;
#pragma unroll
  for (int o = 16; o >= 1; o >>= 1) M = fmaxf(M, __shfl_xor_sync(0xffffffffu, M, o));
  s = m > -INFINITY ? s * expf(m - M) : 0.f;
#pragma unroll
  for (int o = 16; o >= 1; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
  if (lane == 0) sm.stat[warp] = make_float2(M, s);
  // the k-th largest of the warp's g (order32; 0: none)
  auto kth_largest = [&](uint32_t g, uint32_t k) {
    for (; k > 1; --k) {
      const uint32_t top = __reduce_max_sync(0xffffffffu, g);
      if (lane == __ffs(__ballot_sync(0xffffffffu, g == top)) - 1) g = 0;
    }
    return __reduce_max_sync(0xffffffffu, g);
  };
  auto number = [](uint32_t o) { return o > order32(-INFINITY) ? value32(o) : -INFINITY; };
  const uint32_t of_warp = (K + 3) / 4;   // T
  {
    const uint32_t g = kth_largest(order32(m), of_warp);
    if (lane == 0) sm.high[warp] = g;
  }
  __syncthreads();
  const float bound = number(kth_largest(lane < kScanWarps ? sm.high[lane] : 0u, (K + of_warp - 1) / of_warp));
  // ---- list what reaches it.  f(x, index) for every logit that reaches `least` and is not hidden, of
  // the noted sub-blocks, whose words are shared out
  uint16_t* note = sm.note[warp];
  auto read_noted = [&](uint32_t found, float least, auto f) {
    __syncwarp();
    for (uint32_t u = lane; u < 4 * found; u += 32) {
      const int at = note[u >> 2];
      const int g = a0 + (at >> 5) * 128 + (u & 3) * 32 + (at & 31);
      uint4 v = load(g);
      if (next && g < a1) {
        uint4 c = g < whole ? src[g] : hidden;
        for (int n = 0; n < skip; ++n) {
          c = make_uint4(c.y, c.z, c.w, v.x);
          v = make_uint4(v.y, v.z, v.w, 0);
        }
        v = make_uint4(__funnelshift_r(c.x, c.y, shift), __funnelshift_r(c.y, c.z, shift),
                       __funnelshift_r(c.z, c.w, shift), __funnelshift_r(c.w, v.x, shift));
      }
      mend(g, v);
      v = make_uint4(G::clean(v.x), G::clean(v.y), G::clean(v.z), G::clean(v.w));
      typename G::Most mk;
      mk.add(v);
      if (mk.value() < least) continue;
      float x[VEC];
      G::unpack(v, x);
#pragma unroll
      for (int e = 0; e < VEC; ++e)
        if (x[e] >= least && x[e] > -INFINITY) f(x[e], g * VEC + e);
    }
    __syncwarp();
  };
  // of all sub-blocks: the lanes that reach it one after another, a lane for each of their sub-blocks
  auto visit = [&](float least, auto f) {
    uint32_t found = 0;
    for (uint32_t lanes = __ballot_sync(0xffffffffu, m >= least && m > -INFINITY); lanes; lanes &= lanes - 1) {
      const int from = __ffs(lanes) - 1;
      const float mx = lane < subs ? static_cast<float>(sm.most[warp][lane][from]) : -INFINITY;
      const bool in = mx >= least && mx > -INFINITY;
      const uint32_t b = __ballot_sync(0xffffffffu, in);
      if (found + __popc(b) > kNoteMax) {
        read_noted(found, least, f);
        found = 0;
      }
      if (in) note[found + __popc(b & ((1u << lane) - 1u))] = static_cast<uint16_t>(lane * 32 + from);
      found += __popc(b);
    }
    if (found) read_noted(found, least, f);
  };
  uint64_t* out = p.list + static_cast<int64_t>(blockIdx.x) * K;
  visit(bound, [&](float x, int t) {
    const uint32_t k = atomicAdd(&sm.reached, 1);
    if (k < kListMax) sm.list[0][k] = list_key(x, t);
  });
  __syncthreads();
  if (warp == kScanWarps - 1) {
    const float2 st = lane < kScanWarps ? sm.stat[lane] : make_float2(-INFINITY, 0.f);
    float top = st.x;
#pragma unroll
    for (int o = kScanWarps / 2; o >= 1; o >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
    float sum = st.x > -INFINITY ? st.y * expf(st.x - top) : 0.f;
#pragma unroll
    for (int o = kScanWarps / 2; o >= 1; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
    if (lane == 0) p.stat[blockIdx.x] = make_float2(top, sum);
  }
  if (sm.reached <= kListMax) {   // in order (keys differ by their index)
    const uint32_t n = sm.reached;
    if (tid >= n && tid < K) out[tid] = 0;
    if (tid < n) {
      const uint64_t key = sm.list[0][tid];
      uint32_t above = 0;
      for (uint32_t j = 0; j < n; ++j) above += sm.list[0][j] > key;
      if (above < K) out[above] = key;
    }
    return;
  }
  __syncthreads();                // sm.list[0] is the first warp's from here
  // ---- too many: the warp's own K-th largest lane maximum bounds the best K of its part
  const float edge = number(kth_largest(order32(m), K));
  uint64_t* list = sm.list[warp];
  auto put = [&](float x, int t) {
    const uint32_t k = atomicAdd(&sm.count[warp], 1);
    if (k < kListMax) list[k] = list_key(x, t);
  };
  if (M > -INFINITY) visit(edge, put);
  uint32_t n = *static_cast<volatile uint32_t*>(&sm.count[warp]);
  if (n > kListMax) {
    // bisect the K-th largest logit, then, among its equals, the index up to which they count
    auto count_if = [&](float least, auto pred) {
      uint32_t c = 0;
      visit(least, [&](float x, int t) { c += pred(x, t) ? 1u : 0u; });
      return __reduce_add_sync(0xffffffffu, c);
    };
    uint32_t lo = order32(edge), hi = order32(M);   // at least K reach lo
    while (lo < hi) {
      const uint32_t mid = lo + (hi - lo + 1) / 2;
      if (count_if(value32(mid), [](float, int) { return true; }) >= K) lo = mid;
      else hi = mid - 1;
    }
    const float v = value32(lo);
    const uint32_t above = count_if(v, [&](float x, int) { return x > v; });
    int a = 0, b = p.vocab - 1;
    while (a < b) {
      const int mid = a + (b - a) / 2;
      if (count_if(v, [&](float x, int t) { return x == v && t <= mid; }) >= K - above) b = mid;
      else a = mid + 1;
    }
    __syncwarp();
    if (lane == 0) sm.count[warp] = 0;
    __syncwarp();
    visit(v, [&](float x, int t) {
      if (x > v || t <= a) put(x, t);
    });
    n = *static_cast<volatile uint32_t*>(&sm.count[warp]);
  }
  // ---- the warp's best K in order (keys differ by their index), then the CTA's
  uint64_t* best = sm.best + warp * K;
  if (lane >= n && lane < K) best[lane] = 0;
  for (uint32_t i = lane; i < n; i += 32) {
    const uint64_t key = list[i];
    uint32_t above = 0;
    for (uint32_t j = 0; j < n; ++j) above += list[j] > key;
    if (above < K) best[above] = key;
  }
  __syncthreads();
  const uint32_t all = kScanWarps * K;
  if (tid < all) {
    const uint64_t key = sm.best[tid];
    uint32_t above = 0;
    for (uint32_t j = 0; j < all; ++j) above += sm.best[j] > key || (sm.best[j] == key && j < tid);
    if (above < K) out[above] = key;
  }
}

// A sum of two fp32 values, hi + lo with hi the sum's rounding (48 bits or so).
struct TwoFloat {
  float hi, lo;
};
__device__ __forceinline__ TwoFloat two_sum(float a, float b) {   // exact
  const float s = a + b, t = s - a;
  return {s, (a - (s - t)) + (b - t)};
}
__device__ __forceinline__ TwoFloat add(TwoFloat a, float b) {
  const TwoFloat s = two_sum(a.hi, b);
  const float lo = s.lo + a.lo, hi = s.hi + lo;
  return {hi, lo - (hi - s.hi)};
}
// As one number that orders them; 0 is below all.  A sum that left fp32's range (below: a beam's
// score and a difference of logits have it) counts as -inf, and such ones as equal.
__device__ __forceinline__ uint64_t order64(TwoFloat x) {
  const bool fin = fabsf(x.hi) <= FLT_MAX;
  return static_cast<uint64_t>(order32(fin ? x.hi : -INFINITY)) << 32 | order32(fin ? x.lo : 0.f);
}

// log s for s > 0, within about 3e-10: s = 2^e m with m near 1, log m = 2 atanh z = 2 z + R with
// z = (m - 1) / (m + 1), |z| < 0.172; z and e log 2 as two fp32 values each (the first of log 2 has
// 12 bits, so that its product with e is exact), R, below 0.004, by its series in fp32.
__device__ __forceinline__ TwoFloat log_of(TwoFloat s) {
  int e = static_cast<int>(__float_as_uint(s.hi) >> 23) - 127;
  if (__uint_as_float((__float_as_uint(s.hi) & 0x007FFFFFu) | 0x3F800000u) > 1.41421356f) ++e;
  const float down = __uint_as_float(static_cast<uint32_t>(127 - e) << 23);
  const float m = s.hi * down, l = s.lo * down;      // exact
  const float a = m - 1.f;                           // exact
  const TwoFloat d = two_sum(m, 1.f);
  const float z = a / d.hi;
  const float zl = (fmaf(-z, d.hi, a) + l - z * (d.lo + l)) / d.hi;
  const float q = z * z;
  float r = fmaf(q, 2.f / 11, 2.f / 9);
  r = fmaf(q, r, 2.f / 7);
  r = fmaf(q, r, 2.f / 5);
  r = fmaf(q, r, 2.f / 3) * q * z;
  const TwoFloat h = two_sum(e * 0.693115234375f, 2.f * z);
  return add(h, fmaf(static_cast<float>(e), 3.19461849e-5f, 2.f * zl + r) );
}

// One CTA per request.  Shared memory: the totals (order64) and candidates ~(i, t) of its beams'
// segments, segment after segment, best first, and the segments' heads.
constexpr int merge_smem_bytes(int beams, int splits) {
  return beams * splits * (12 * beams + 2);
}
// The most of any call: one request whose segments were halved once more while it had fewer than 304
constexpr int merge_smem_most() {
  int most = 0;
  for (int k = 1; k <= kMaxBeams; ++k) {
    const int bytes = merge_smem_bytes(k, 2 * (kBeamMinSegments - 1) / k);
    if (bytes > most) most = bytes;
  }
  return most;
}
static_assert(merge_smem_most() + 2048 <= 227 * 1024, "dynamic and static shared memory of the merge");
template <class T>
__global__ void __launch_bounds__(kMergeThreads) beam_merge_kernel(const BeamParams p) {
  extern __shared__ __align__(16) uint8_t merge_smem[];
  __shared__ float most[32], last[32], score[32];   // the row's largest logit; the one of eos
  __shared__ TwoFloat log_sum[32];
  __shared__ uint64_t best_total[32], end_total[32];
  __shared__ uint32_t best_at[32];
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int K = p.beams, NL = K * p.splits, N = NL * K;
  const int64_t b = blockIdx.x;
  uint64_t* total = reinterpret_cast<uint64_t*>(merge_smem);
  uint32_t* cand = reinterpret_cast<uint32_t*>(total + N);
  uint16_t* head = reinterpret_cast<uint16_t*>(cand + N);       // a list's first not taken
  const T* logits = static_cast<const T*>(p.logits) + b * K * p.vocab;
  griddep_wait();
  griddep_launch();
  const float2* stat = p.stat + b * NL;
  const uint64_t* list = p.list + b * N;
  for (int k = tid; k < N; k += kMergeThreads) total[k] = list[k];
  // a warp per beam: the maximum and the sum of its segments and of the logit that ends it
  int width = 1;                                     // lanes with a segment, as a power of two
  while (width < 32 && width < p.splits) width *= 2;
  for (int i = warp; i < K; i += kMergeThreads / 32) {
    const float c = p.scores[b * K + i];
    const float x = p.eos >= 0 ? Logits<T>::one(logits[static_cast<int64_t>(i) * p.vocab + p.eos])
                               : -INFINITY;
    const float2 none = make_float2(-INFINITY, 0.f);
    const float2 st0 = lane < p.splits ? stat[i * p.splits + lane] : none;
    float m = fmaxf(x, st0.x);
    for (int k = lane + 32; k < p.splits; k += 32) m = fmaxf(m, stat[i * p.splits + k].x);
    for (int o = width / 2; o >= 1; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
    TwoFloat s{0.f, 0.f};                            // (lanes from width on: not taken)
    if (lane < width && m > -INFINITY) {
      s.hi = st0.y * expf(st0.x - m);
      if (lane == 0) s = add(s, expf(x - m));
      for (int k = lane + 32; k < p.splits; k += 32) {
        const float2 st = stat[i * p.splits + k];
        s = add(s, st.y * expf(st.x - m));
      }
    }
    for (int o = width / 2; o >= 1; o >>= 1) {
      const float h = __shfl_xor_sync(0xffffffffu, s.hi, o), l = __shfl_xor_sync(0xffffffffu, s.lo, o);
      s = add(s, h);
      s.lo += l;
    }
    if (lane == 0) {
      log_sum[i] = m > -INFINITY ? log_of(s) : TwoFloat{0.f, 0.f};
      most[i] = m;
      last[i] = x;
      score[i] = c;
    }
  }
  for (int l = tid; l < NL; l += kMergeThreads) head[l] = 0;
  __syncthreads();
  // (x - M) - log sum + c; 0: no candidate (a dead beam, a hidden logit)
  auto total_of = [&](int i, float x) -> uint64_t {
    const float c = score[i];
    if (!(fabsf(c) <= FLT_MAX) || !(x > -INFINITY)) return 0;
    TwoFloat t = two_sum(x, -most[i]);
    t = add(t, -log_sum[i].hi);
    t = add(t, -log_sum[i].lo);
    return order64(add(t, c));
  };
  for (int k = tid; k < N; k += kMergeThreads) {
    const uint64_t key = total[k];
    const int i = k / (p.splits * K);
    total[k] = key ? total_of(i, value32(static_cast<uint32_t>(key >> 32))) : 0;
    cand[k] = ~(static_cast<uint32_t>(i) * p.vocab + ~static_cast<uint32_t>(key));
  }
  if (tid < K) end_total[tid] = p.eos >= 0 ? total_of(tid, last[tid]) : 0;
  __syncthreads();
  if (warp != 0) return;
  // best first: every lane holds the first in order (larger total, then lower (i, t)) of its
  // lists' heads; the warp takes the first of them K times
  uint64_t first = 0;
  uint32_t first_at = 0;
  int first_list = -1;
  auto look = [&]() {
    first = 0;
    first_at = 0;
    for (int l = lane; l < NL; l += 32) {
      const int k = head[l];
      if (k == K) continue;
      const uint64_t t = total[l * K + k];
      const uint32_t a = cand[l * K + k];
      if (t > first || (t == first && t != 0 && a > first_at)) {
        first = t;
        first_at = a;
        first_list = l;
      }
    }
  };
  look();
  for (int r = 0; r < K; ++r) {
    const uint32_t hi = __reduce_max_sync(0xffffffffu, static_cast<uint32_t>(first >> 32));
    const uint32_t lo = __reduce_max_sync(
        0xffffffffu, static_cast<uint32_t>(first >> 32) == hi ? static_cast<uint32_t>(first) : 0u);
    const uint64_t top = static_cast<uint64_t>(hi) << 32 | lo;
    const uint32_t a = __reduce_max_sync(0xffffffffu, first == top ? first_at : 0u);
    if (lane == 0) {
      best_total[r] = top;
      best_at[r] = ~a;
    }
    if (top != 0 && first == top && first_at == a) {   // at most one lane: candidates differ
      ++head[first_list];
      look();
    }
  }
  __syncwarp();
  auto value = [](uint64_t o) { return value32(static_cast<uint32_t>(o >> 32)); };
  if (lane < K) {
    const bool any = best_total[lane] != 0;
    const uint32_t at = best_at[lane];
    const int i = any ? static_cast<int>(at / static_cast<uint32_t>(p.vocab)) : 0;
    p.next_scores[b * K + lane] = any ? value(best_total[lane]) : -INFINITY;
    p.tokens[b * K + lane] = any ? static_cast<int32_t>(at - static_cast<uint32_t>(i) * p.vocab) : -1;
    p.parents[b * K + lane] = any ? static_cast<int32_t>(b * K + i) : -1;
    if (p.ended != nullptr) {
      // candidates before (lane, eos): of the best K, and the other beams' ends
      const uint64_t mine = end_total[lane];
      const uint32_t me = static_cast<uint32_t>(lane) * p.vocab + p.eos;
      int before = 0;
      for (int r = 0; r < K; ++r) {
        before += best_total[r] > mine || (best_total[r] == mine && best_at[r] < me);
        before += end_total[r] > mine || (end_total[r] == mine && r < lane);
      }
      p.ended[b * K + lane] = mine != 0 && before < K ? value(mine) : -INFINITY;
    }
  }
}

template <class T>
static cudaError_t launch_beam_type(const BeamParams& p, cudaStream_t s) {
  cudaError_t e = launch_pdl(beam_scan_kernel<T>,
                             dim3(static_cast<unsigned>(p.batch) * p.beams * p.splits),
                             dim3(kScanThreads), 0, s, true, p);
  if (e != cudaSuccess) return e;
  const int smem = merge_smem_bytes(p.beams, p.splits);
  // the limit is the function's, whichever thread launches it: always the same one, so that no call
  // lowers it between another's request and launch
  if (smem > 48 * 1024 &&
      (e = cudaFuncSetAttribute(beam_merge_kernel<T>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                merge_smem_most())) != cudaSuccess)
    return e;
  return launch_pdl(beam_merge_kernel<T>, dim3(p.batch), dim3(kMergeThreads), smem, s, true, p);
}

cudaError_t launch_beam_select(const BeamParams& p, int dtype, cudaStream_t s) {
  if (dtype == RCP_LOGITS_FP16) return launch_beam_type<__half>(p, s);
  if (dtype == RCP_LOGITS_BF16) return launch_beam_type<__nv_bfloat16>(p, s);
  return launch_beam_type<float>(p, s);
}

}  // namespace rcp
