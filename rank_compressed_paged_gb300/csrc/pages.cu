// Data movement of the page pool: page copies (copy-on-write of forked sequences) and the
// in-place compaction of a request's kept tokens.  Both move bytes only, whatever the page
// format holds, and are bounded by HBM: every moved byte is read once and written once.
#include <cuda_runtime.h>

#include <cstdint>

#include "launch.h"
#include "ptx.cuh"
#include "rcp.h"
#include "shape.h"

namespace rcp {

// Bytes of one token row and one page of a cache.
template <class S, int FMT>
struct PageGeom {
  static constexpr bool I4 = FMT == RCP_PAGES_INT4;
  static constexpr int KROW = I4 ? S::RK / 2 : FMT == RCP_PAGES_FP8_E4M3 ? S::RK : S::RK * 2;
  static constexpr int VROW = I4 ? S::R / 2 : FMT == RCP_PAGES_FP8_E4M3 ? S::R : S::R * 2;
  static constexpr int KCODES = S::H * kBlockSize * KROW;   // before the 4-bit pages' scales
  static constexpr int VCODES = kBlockSize * VROW;
  static constexpr int KP = KCODES + (I4 ? S::H * kBlockSize * 2 : 0);
  static constexpr int VP = VCODES + (I4 ? kBlockSize * (S::R / 64) * 2 : 0);
  static_assert(KP % 16 == 0 && VP % 16 == 0, "16-byte copies");
};

// ------------------------------------------------------------------------------ page copies
constexpr int kCopyThreads = 128;
constexpr int kCopyUnroll = 4;   // 16-byte words per thread, all loads before the first store

// Destinations of a copy whose source is one page, passed by value (N = 1: none, the pairs are
// on the device).
template <int N>
struct CopyList {
  int32_t dst[N];
};

template <class S, int FMT, int N>
__global__ void __launch_bounds__(kCopyThreads)
    copy_pages_kernel(const CopyParams p, const __grid_constant__ CopyList<N> list) {
  using G = PageGeom<S, FMT>;
  constexpr int KU = G::KP / 16, U = (G::KP + G::VP) / 16;
  constexpr int PER = kCopyThreads * kCopyUnroll, PIECES = (U + PER - 1) / PER;
  griddep_wait();   // the pages (and the pairs) may come from the launch before
  griddep_launch();
  const int64_t total = static_cast<int64_t>(p.n) * PIECES;
  for (int64_t w = blockIdx.x; w < total; w += gridDim.x) {
    const int i = static_cast<int>(w / PIECES), piece = static_cast<int>(w % PIECES);
    int64_t src = p.src, dst;
    if constexpr (N > 1) {
      dst = list.dst[i];
    } else {
      src = p.pairs[2 * static_cast<int64_t>(i)];
      dst = p.pairs[2 * static_cast<int64_t>(i) + 1];
    }
    if (src == -1 || dst == -1) continue;   // padding
    if (src < 0 || src >= p.num_blocks || dst < 0 || dst >= p.num_blocks) {
      if (threadIdx.x == 0) atomicOr(p.dev_err, RCP_DEVERR_BAD_BLOCK);
      continue;
    }
    const uint4* ks = reinterpret_cast<const uint4*>(static_cast<uint8_t*>(p.k_pages) + src * G::KP);
    const uint4* vs = reinterpret_cast<const uint4*>(static_cast<uint8_t*>(p.v_pages) + src * G::VP);
    uint4* kd = reinterpret_cast<uint4*>(static_cast<uint8_t*>(p.k_pages) + dst * G::KP);
    uint4* vd = reinterpret_cast<uint4*>(static_cast<uint8_t*>(p.v_pages) + dst * G::VP);
    uint4 r[kCopyUnroll];
    const int u0 = piece * PER + threadIdx.x;
#pragma unroll
    for (int k = 0; k < kCopyUnroll; ++k) {
      const int u = u0 + k * kCopyThreads;
      if (u < U) r[k] = u < KU ? ks[u] : vs[u - KU];
    }
#pragma unroll
    for (int k = 0; k < kCopyUnroll; ++k) {
      const int u = u0 + k * kCopyThreads;
      if (u < U) *(u < KU ? kd + u : vd + (u - KU)) = r[k];
    }
  }
}

// -------------------------------------------------------------------------------- compaction
// Kept token number j of a request moves to table position j, in place.  A token never moves
// up (j <= its position), which gives the order: a CTA owns some bytes of every token of one
// request (a slice) and goes through the kept tokens in windows, loading a whole window into
// registers before it stores it.  A store then only hits positions whose own tokens were
// loaded in this window or an earlier one.  Slices and requests never share a byte, so no CTA
// waits for another.
constexpr int kCmpThreads = 256;
constexpr int kCmpSpan = kCmpThreads * 8;      // mask bytes scanned at a time
constexpr int kCmpPages = kCmpSpan / kBlockSize;
constexpr int kCmpUnroll = 4;                  // words per thread and window
constexpr int kSliceBytes = 64;                // bytes of a token row per slice

// One slice: unit u of a token (VT-sized) at
//   base + page * page_stride + (token % 16) * row_stride + (u >> upr) * group + (u % 2^upr) * sizeof(VT)
struct Slice {
  uint8_t* base;
  int64_t page_stride;
  int32_t row_stride, group;
  int32_t upr;      // log2 units per row piece
  int32_t units;    // log2 units per token
};

struct CompactSmem {
  uint16_t src[kCmpSpan];              // kept tokens of the span, relative to its start
  int32_t spage[kCmpPages];            // the span's pages
  int32_t dpage[kCmpPages + 1];        // pages of its destinations
  int32_t wsum[kCmpThreads / 32];
};

// Moves the span's `count` kept tokens: token i from position s0 + src[i] to d0 + i, unless
// that is where it is (a page whose tokens all stay is not written: it may be shared).
template <class VT, bool TOKEN_FIRST>
__device__ __forceinline__ void move_span(const Slice& sl, const CompactSmem& sm, int count, int s0,
                                          int d0, uint32_t* dev_err) {
  const int items = count << sl.units;
  const int umask = (1 << sl.units) - 1, rmask = (1 << sl.upr) - 1;
  // item -> (token, unit): units fastest (whole rows), or tokens fastest when a row piece is
  // smaller than a word and a page keeps the pieces of its tokens side by side
  auto split = [&](int it, int& i, int& u) {
    if (TOKEN_FIRST) {
      u = (it >> 4) & umask;
      i = ((it >> (4 + sl.units)) << 4) | (it & 15);
    } else {
      i = it >> sl.units;
      u = it & umask;
    }
  };
  const int span = TOKEN_FIRST ? ((count + 15) & ~15) << sl.units : items;
  auto at = [&](int64_t page, int off, int u) {
    return reinterpret_cast<VT*>(sl.base + page * sl.page_stride + off * sl.row_stride +
                                 (u >> sl.upr) * sl.group) + (u & rmask);
  };
  constexpr int PER = kCmpThreads * kCmpUnroll;
  VT cur[kCmpUnroll], nxt[kCmpUnroll];
  auto load = [&](VT (&r)[kCmpUnroll], int w0) {
#pragma unroll
    for (int k = 0; k < kCmpUnroll; ++k) {
      const int it = w0 + k * kCmpThreads + threadIdx.x;
      int i, u;
      split(it, i, u);
      if (it < span && i < count) {
        const int s = sm.src[i];
        const int page = sm.spage[s / kBlockSize];
        if (s0 + s == d0 + i) continue;
        if (page >= 0) r[k] = *at(page, s % kBlockSize, u);
        else atomicOr(dev_err, RCP_DEVERR_BAD_BLOCK);
      }
    }
  };
  auto store = [&](const VT (&r)[kCmpUnroll], int w0) {
#pragma unroll
    for (int k = 0; k < kCmpUnroll; ++k) {
      const int it = w0 + k * kCmpThreads + threadIdx.x;
      int i, u;
      split(it, i, u);
      if (it < span && i < count) {
        const int d = d0 % kBlockSize + i, s = sm.src[i];
        const int page = sm.dpage[d / kBlockSize];
        if (s0 + s == d0 + i) continue;
        if (page >= 0) {
          if (sm.spage[s / kBlockSize] >= 0) *at(page, d % kBlockSize, u) = r[k];
        } else {
          atomicOr(dev_err, RCP_DEVERR_BAD_BLOCK);
        }
      }
    }
  };
  load(cur, 0);
  for (int w0 = 0; w0 < span; w0 += PER) {
    if (w0 + PER < span) load(nxt, w0 + PER);
    __syncthreads();   // every thread has loaded this window
    store(cur, w0);
#pragma unroll
    for (int k = 0; k < kCmpUnroll; ++k) cur[k] = nxt[k];
  }
}

template <class S, int FMT>
struct CompactSlices {
  using G = PageGeom<S, FMT>;
  // a key slice: one piece of a head's row, or several heads' whole rows
  static constexpr int KPIECE = G::KROW < kSliceBytes ? G::KROW : kSliceBytes;
  static constexpr int KPARTS = G::KROW / KPIECE;
  static constexpr int KHEADS = kSliceBytes / KPIECE < S::H ? kSliceBytes / KPIECE : S::H;
  static constexpr int NK = S::H / KHEADS * KPARTS;
  static constexpr int VPIECE = G::VROW < kSliceBytes ? G::VROW : kSliceBytes;
  static constexpr int NV = G::VROW / VPIECE;
  static constexpr int N = NK + NV + (G::I4 ? 2 : 0);
};

constexpr int log2i(int x) { return x <= 1 ? 0 : 1 + log2i(x / 2); }

template <class S, int FMT>
__global__ void __launch_bounds__(kCmpThreads) compact_kernel(const CompactParams p) {
  using G = PageGeom<S, FMT>;
  using C = CompactSlices<S, FMT>;
  __shared__ CompactSmem sm;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int b = blockIdx.x / C::N, slice = blockIdx.x % C::N;
  griddep_wait();   // the pages, lengths and mask may come from the launch before
  griddep_launch();
  const int32_t max_len = p.bt_stride * kBlockSize;
  int32_t L = p.seq_lens[b];
  if (L < 0 || L > max_len) {
    if (slice == 0 && tid == 0) atomicOr(p.dev_err, RCP_DEVERR_BAD_LEN);
    L = 0;
  }
  uint8_t* kp = static_cast<uint8_t*>(p.k_pages);
  uint8_t* vp = static_cast<uint8_t*>(p.v_pages);
  const int32_t* table = p.block_table + static_cast<int64_t>(b) * p.bt_stride;
  const uint8_t* keep = p.keep + static_cast<int64_t>(b) * max_len;
  constexpr int KVT = C::KPIECE < 16 ? C::KPIECE : 16;   // word of a key slice
  Slice sl;
  if (slice < C::NK) {
    const int part = slice % C::KPARTS, h0 = slice / C::KPARTS * C::KHEADS;
    sl = Slice{kp + h0 * kBlockSize * G::KROW + part * C::KPIECE, G::KP, G::KROW,
               kBlockSize * G::KROW, log2i(C::KPIECE / KVT), log2i(C::KHEADS * C::KPIECE / KVT)};
  } else if (slice < C::NK + C::NV) {
    sl = Slice{vp + (slice - C::NK) * C::VPIECE, G::VP, G::VROW, 0, log2i(C::VPIECE / 16),
               log2i(C::VPIECE / 16)};
  } else if (slice == C::NK + C::NV) {   // key scales: [H][16] fp16
    sl = Slice{kp + G::KCODES, G::KP, 2, kBlockSize * 2, 0, log2i(S::H)};
  } else {                               // value scales: [16][R / 64] fp16
    sl = Slice{vp + G::VCODES, G::VP, S::R / 64 * 2, 0, log2i(S::R / 64), log2i(S::R / 64)};
  }
  int d0 = 0;   // kept tokens so far
  for (int s0 = 0; s0 < L; s0 += kCmpSpan) {
    __syncthreads();   // the previous span's lists are no longer read
    // this thread's eight mask bytes as bits, tokens past the end dropped
    uint32_t bits = 0;
    const int t0 = s0 + tid * 8;
    if (t0 < L) {
      const uint2 m = *reinterpret_cast<const uint2*>(keep + t0);
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        if ((m.x >> (8 * e)) & 0xFFu) bits |= 1u << e;
        if ((m.y >> (8 * e)) & 0xFFu) bits |= 16u << e;
      }
      if (L - t0 < 8) bits &= (1u << (L - t0)) - 1u;
    }
    int incl = __popc(bits);
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int y = __shfl_up_sync(0xffffffffu, incl, o);
      if (lane >= o) incl += y;
    }
    if (lane == 31) sm.wsum[warp] = incl;
    __syncthreads();
    int count = 0, first = incl - __popc(bits);
#pragma unroll
    for (int w = 0; w < kCmpThreads / 32; ++w) {
      if (w < warp) first += sm.wsum[w];
      count += sm.wsum[w];
    }
    const int span = L - s0 < kCmpSpan ? L - s0 : kCmpSpan;
    if (d0 == s0 && count == span) {   // nothing dropped so far: every token is in its place
      d0 += count;
      continue;
    }
    for (uint32_t m = bits; m != 0; m &= m - 1)
      sm.src[first++] = static_cast<uint16_t>(tid * 8 + __ffs(m) - 1);
    auto page_of = [&](int j) {
      const int32_t id = table[j];
      return id >= 0 && id < p.num_blocks ? id : -1;
    };
    for (int j = tid; j < (span + kBlockSize - 1) / kBlockSize; j += kCmpThreads)
      sm.spage[j] = page_of(s0 / kBlockSize + j);
    const int dn = count > 0 ? (d0 % kBlockSize + count + kBlockSize - 1) / kBlockSize : 0;
    for (int j = tid; j < dn; j += kCmpThreads) sm.dpage[j] = page_of(d0 / kBlockSize + j);
    __syncthreads();
    if (count > 0) {
      if (slice < C::NK) {
        if constexpr (KVT == 16) move_span<uint4, false>(sl, sm, count, s0, d0, p.dev_err);
        else move_span<uint2, false>(sl, sm, count, s0, d0, p.dev_err);
      } else if (slice < C::NK + C::NV) {
        move_span<uint4, false>(sl, sm, count, s0, d0, p.dev_err);
      } else if constexpr (G::I4) {
        if (slice == C::NK + C::NV) move_span<uint16_t, true>(sl, sm, count, s0, d0, p.dev_err);
        else move_span<uint16_t, false>(sl, sm, count, s0, d0, p.dev_err);
      }
    }
    d0 += count;
  }
  if (slice == 0 && tid == 0) p.new_lens[b] = d0;
}

// --------------------------------------------------------------------------------- launches
template <class S, int FMT>
cudaError_t copy_pages_fmt(const CopyParams& p, const int32_t* list, int num_sms,
                           cudaStream_t stream) {
  using G = PageGeom<S, FMT>;
  constexpr int PER = kCopyThreads * kCopyUnroll;
  constexpr int PIECES = ((G::KP + G::VP) / 16 + PER - 1) / PER;
  const int64_t total = static_cast<int64_t>(p.n) * PIECES, cap = static_cast<int64_t>(num_sms) * 64;
  const dim3 grid(static_cast<unsigned>(total < cap ? total : cap));
  if (p.pairs) {
    const CopyList<1> none{};
    return launch_pdl(copy_pages_kernel<S, FMT, 1>, grid, dim3(kCopyThreads), 0, stream, true, p,
                      none);
  }
  CopyList<kCopyListMax> l;
  for (int i = 0; i < p.n; ++i) l.dst[i] = list[i];
  return launch_pdl(copy_pages_kernel<S, FMT, kCopyListMax>, grid, dim3(kCopyThreads), 0, stream,
                    true, p, l);
}

template <class S>
cudaError_t launch_copy_pages(const CopyParams& p, const int32_t* list, int page_format,
                              int num_sms, cudaStream_t stream) {
  if (page_format == RCP_PAGES_FP8_E4M3)
    return copy_pages_fmt<S, RCP_PAGES_FP8_E4M3>(p, list, num_sms, stream);
  if (page_format == RCP_PAGES_INT4)
    return copy_pages_fmt<S, RCP_PAGES_INT4>(p, list, num_sms, stream);
  return copy_pages_fmt<S, RCP_PAGES_FP16>(p, list, num_sms, stream);
}

template <class S, int FMT>
cudaError_t compact_fmt(const CompactParams& p, cudaStream_t stream) {
  return launch_pdl(compact_kernel<S, FMT>,
                    dim3(static_cast<unsigned>(p.batch) * CompactSlices<S, FMT>::N),
                    dim3(kCmpThreads), 0, stream, true, p);
}

template <class S>
cudaError_t launch_compact(const CompactParams& p, int page_format, cudaStream_t stream) {
  if (page_format == RCP_PAGES_FP8_E4M3) return compact_fmt<S, RCP_PAGES_FP8_E4M3>(p, stream);
  if (page_format == RCP_PAGES_INT4) return compact_fmt<S, RCP_PAGES_INT4>(p, stream);
  return compact_fmt<S, RCP_PAGES_FP16>(p, stream);
}

template cudaError_t launch_copy_pages<ShapeMain>(const CopyParams&, const int32_t*, int, int,
                                                  cudaStream_t);
template cudaError_t launch_copy_pages<ShapeTiny>(const CopyParams&, const int32_t*, int, int,
                                                  cudaStream_t);
template cudaError_t launch_compact<ShapeMain>(const CompactParams&, int, cudaStream_t);
template cudaError_t launch_compact<ShapeTiny>(const CompactParams&, int, cudaStream_t);

}  // namespace rcp
