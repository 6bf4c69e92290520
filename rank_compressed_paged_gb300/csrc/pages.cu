// Data movement of the page pool: page copies (copy-on-write of forked sequences) and the
// in-place compaction of a request's kept tokens.  Both move bytes only, whatever the page
// format holds, and are bounded by HBM: every moved byte is read once and written once.
#include <cuda_runtime.h>

#include <cstdint>
#include <type_traits>

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
// A CTA copies 8 KB pieces (four 16-byte words per thread, all loads ahead of the stores): 4096
// fp16 pages of 98 KB in 120 us, 6.7 TB/s, 0.99 of the copy rate.  One page is a launch.
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
// up (j <= its position), which gives the order: a cluster of CTAs owns some bytes of every
// token of one request (a slice) and goes through the kept tokens in windows; its CTAs load
// the whole window into registers, meet at the cluster's barrier, and store it (another CTA
// of the SM loads meanwhile).  A store only hits positions whose own tokens were
// loaded in this window or an earlier one.  Slices and requests never share a byte, so no
// cluster waits for another.
//
// Bound by HBM: moved bytes read once and written once, the mask read by every CTA of its
// request (from L2).  Slices of 128 to 256 bytes keep whole rows together.  Measured, half of
// 64 x 8192 tokens kept: fp16 370 us (6.4 TB/s, 0.94 of the copy rate), E4M3 217 us (5.5),
// 4-bit 146 us (4.3: a kept token's key rows are 32-byte pieces, of 64-byte memory accesses);
// 0.6 of one 30001-token request: 69, 36 and 32 us (the 4-bit one 35 with the pages out of L2),
// of which the scan of the mask and the list take 7; there a window costs the latency of its
// loads plus the cluster's barrier, whose ordering of memory costs 1 to 3 us of them.
// (Slices of 64 bytes and one CTA each, the first form, took 644 us and, with all 4-bit key
// scales in one slice, 909 us for the single request.)
constexpr int kCmpThreads = 512;
constexpr int kCmpQuarter = kCmpThreads * 16;  // mask bytes a thread group scans in one load
constexpr int kCmpSpan = kCmpQuarter * 4;      // ... and at a time
constexpr int kCmpPages = kCmpSpan / kBlockSize;
constexpr int kCmpUnroll = 4;                  // words per thread and window
constexpr int kCmpCluster = 8;                 // CTAs per slice at most

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
  uint64_t wsum[kCmpThreads / 32];     // a warp's kept tokens, 16 bits per quarter
  int32_t moved;                       // first kept token of the span that moves
};

// Moves kept tokens first .. count - 1 of a span: token i from position s0 + src[i] to d0 + i,
// all of them above their destination (a page whose tokens all stay is not written: it may
// be shared).
template <class VT, bool TOKEN_FIRST, bool CLUSTER>
__device__ __forceinline__ void move_span(const Slice& sl, CompactSmem& sm, int first,
                                          int count, int d0, int rank, int ctas, uint32_t* dev_err) {
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
  const int begin = (TOKEN_FIRST ? first & ~15 : first) << sl.units;
  const int end = (TOKEN_FIRST ? (count + 15) & ~15 : count) << sl.units;
  auto at = [&](int page, int off, int u) {
    return reinterpret_cast<VT*>(sl.base + page * sl.page_stride + off * sl.row_stride +
                                 (u >> sl.upr) * sl.group) + (u & rmask);
  };
  constexpr int UNR = kCmpUnroll, PER = kCmpThreads * UNR;   // items of a CTA's share of a window
  const int dof = d0 % kBlockSize;
  bool bad = false;
  for (int w0 = begin; w0 < end; w0 += PER * ctas) {
    const int mine = w0 + rank * PER + static_cast<int>(threadIdx.x);
    VT r[UNR] = {};
#pragma unroll
    for (int k = 0; k < UNR; ++k) {
      int i, u;
      split(mine + k * kCmpThreads, i, u);
      if (i < count && (!TOKEN_FIRST || i >= first)) {
        const int s = sm.src[i], page = sm.spage[s / kBlockSize];
        if (page >= 0) r[k] = *at(page, s % kBlockSize, u);
        else bad = true;
      }
    }
    // every thread of the cluster has loaded this window, before any of them stores it: the
    // barrier releases and acquires, which orders other threads' stores behind these loads
    if (CLUSTER) cluster_sync_all();
    else __syncthreads();
#pragma unroll
    for (int k = 0; k < UNR; ++k) {
      int i, u;
      split(mine + k * kCmpThreads, i, u);
      if (i < count && (!TOKEN_FIRST || i >= first)) {
        const int d = dof + i, page = sm.dpage[d / kBlockSize];
        const bool loaded = sm.spage[sm.src[i] / kBlockSize] >= 0;
        if (page >= 0 && loaded) *at(page, d % kBlockSize, u) = r[k];
        bad |= page < 0;
      }
    }
  }
  if (bad) atomicOr(dev_err, RCP_DEVERR_BAD_BLOCK);
}

template <class S, int FMT, bool CLUSTER>
struct CompactSlices {
  using G = PageGeom<S, FMT>;
  // bytes of a token row: 24 slices of equal size (4-bit pages: 17, with the scales' own)
  static constexpr int BYTES = FMT == RCP_PAGES_FP16 ? 256 : G::I4 && CLUSTER ? 64 : 128;
  // a key slice: several heads' rows; 4-bit key scales: eight heads', two bytes each
  static constexpr int KHEADS = BYTES / G::KROW < S::H ? BYTES / G::KROW : S::H;
  static constexpr int NK = S::H / KHEADS;
  static constexpr int VPIECE = G::VROW < BYTES ? G::VROW : BYTES;
  static constexpr int NV = G::VROW / VPIECE;
  static constexpr int SHEADS = S::H < 8 ? S::H : 8;
  static constexpr int NS = G::I4 ? S::H / SHEADS : 0;
  static constexpr int N = NK + NV + NS + (G::I4 ? 1 : 0);
  static_assert(BYTES % G::KROW == 0 && S::H % KHEADS == 0 && G::VROW % VPIECE == 0, "slices");
};

using False = std::false_type;
using True = std::true_type;
constexpr int log2i(int x) { return x <= 1 ? 0 : 1 + log2i(x / 2); }

template <class S, int FMT, bool CLUSTER>
__global__ void __launch_bounds__(kCmpThreads, 2) compact_kernel(const CompactParams p) {
  using G = PageGeom<S, FMT>;
  using C = CompactSlices<S, FMT, CLUSTER>;
  extern __shared__ __align__(16) uint8_t smem_raw[];
  CompactSmem& sm = *reinterpret_cast<CompactSmem*>(smem_raw);
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int rank = CLUSTER ? blockIdx.x % p.ctas : 0;   // of the slice's cluster
  const int unit = CLUSTER ? blockIdx.x / p.ctas : blockIdx.x;
  const int b = unit / C::N, slice = unit % C::N;
  griddep_wait();   // the pages, lengths and mask may come from the launch before
  griddep_launch();
  const int32_t max_len = p.bt_stride * kBlockSize;
  int32_t L = p.seq_lens[b];
  if (L < 0 || L > max_len) {
    if (slice == 0 && rank == 0 && tid == 0) atomicOr(p.dev_err, RCP_DEVERR_BAD_LEN);
    L = 0;
  }
  uint8_t* kp = static_cast<uint8_t*>(p.k_pages);
  uint8_t* vp = static_cast<uint8_t*>(p.v_pages);
  const int32_t* table = p.block_table + static_cast<int64_t>(b) * p.bt_stride;
  const uint8_t* keep = p.keep + static_cast<int64_t>(b) * max_len;
  constexpr int KVT = G::KROW < 16 ? G::KROW : 16;       // word of a key slice
  constexpr int VSC = S::R / 64 * 2;                     // a token's value scales
  constexpr int VSVT = VSC < 16 ? 2 : 16;
  Slice sl;
  if (slice < C::NK) {
    sl = Slice{kp + slice * C::KHEADS * kBlockSize * G::KROW, G::KP, G::KROW, kBlockSize * G::KROW,
               log2i(G::KROW / KVT), log2i(C::KHEADS * G::KROW / KVT)};
  } else if (slice < C::NK + C::NV) {
    sl = Slice{vp + (slice - C::NK) * C::VPIECE, G::VP, G::VROW, 0, log2i(C::VPIECE / 16),
               log2i(C::VPIECE / 16)};
  } else if (slice < C::NK + C::NV + C::NS) {   // key scales: [H][16] fp16
    sl = Slice{kp + G::KCODES + (slice - C::NK - C::NV) * C::SHEADS * kBlockSize * 2, G::KP, 2,
               kBlockSize * 2, 0, log2i(C::SHEADS)};
  } else {                                      // value scales: [16][R / 64] fp16
    sl = Slice{vp + G::VCODES, G::VP, VSC, 0, log2i(VSC / VSVT), log2i(VSC / VSVT)};
  }
  int d0 = 0;   // kept tokens so far
  for (int s0 = 0; s0 < L; s0 += kCmpSpan) {
    __syncthreads();   // the previous span's lists are no longer read
    // mask bytes as bits, tokens past the end dropped: thread t has the 16 tokens from 16 t on
    // of every quarter of the span; the quarters' counts are scanned as one packed word
    uint32_t bits[4];
    uint64_t mine = 0;
#pragma unroll
    for (int q = 0; q < 4; ++q) {
      const int t0 = s0 + q * kCmpQuarter + tid * 16;
      bits[q] = 0;
      if (t0 < L) {
        const uint4 m = *reinterpret_cast<const uint4*>(keep + t0);
        const uint32_t w[4] = {m.x, m.y, m.z, m.w};
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          // a byte's highest bit set iff the byte is not zero, then the four gathered
          const uint32_t nz = (((w[e] & 0x7F7F7F7Fu) + 0x7F7F7F7Fu) | w[e]) & 0x80808080u;
          bits[q] |= (((nz >> 7) * 0x01020408u) >> 24 & 0xFu) << (4 * e);
        }
        if (L - t0 < 16) bits[q] &= (1u << (L - t0)) - 1u;
      }
      mine |= static_cast<uint64_t>(__popc(bits[q])) << (16 * q);
    }
    uint64_t incl = mine;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const uint64_t y = __shfl_up_sync(0xffffffffu, incl, o);
      if (lane >= o) incl += y;
    }
    if (lane == 31) sm.wsum[warp] = incl;
    if (tid == 0) sm.moved = kCmpSpan;
    __syncthreads();
    uint64_t first = incl - mine, total = 0;   // per quarter
#pragma unroll
    for (int w = 0; w < kCmpThreads / 32; ++w) {
      if (w < warp) first += sm.wsum[w];
      total += sm.wsum[w];
    }
    auto page_of = [&](int j) {
      const int32_t id = table[j];
      return id >= 0 && id < p.num_blocks ? id : -1;
    };
    const int span = L - s0 < kCmpSpan ? L - s0 : kCmpSpan;
    for (int j = tid; j < (span + kBlockSize - 1) / kBlockSize; j += kCmpThreads)
      sm.spage[j] = page_of(s0 / kBlockSize + j);
    // the list, 32 tokens at a time: lane e takes token e of the bits of a pair of lanes, so
    // that a warp's stores are side by side
    int moved = kCmpSpan, count = 0;
    for (int q = 0; q * kCmpQuarter < span; ++q) {
      const int mybits = static_cast<int>(q < 2 ? (q == 0 ? bits[0] : bits[1]) : (q == 2 ? bits[2] : bits[3]));
      const int mystart = count + static_cast<int>((first >> (16 * q)) & 0xFFFFu);
#pragma unroll 4
      for (int pair = 0; pair < 16; ++pair) {
        const uint32_t w = static_cast<uint32_t>(__shfl_sync(0xffffffffu, mybits, 2 * pair)) |
                           static_cast<uint32_t>(__shfl_sync(0xffffffffu, mybits, 2 * pair + 1)) << 16;
        const int at = __shfl_sync(0xffffffffu, mystart, 2 * pair);
        if ((w >> lane) & 1u) {
          const int i = at + __popc(w & ((1u << lane) - 1u));
          const int s = q * kCmpQuarter + (warp * 16 + pair) * 32 + lane;
          sm.src[i] = static_cast<uint16_t>(s);
          if (s0 + s != d0 + i && i < moved) moved = i;
        }
      }
      count += static_cast<int>((total >> (16 * q)) & 0xFFFFu);
    }
    const int dn = count > 0 ? (d0 % kBlockSize + count + kBlockSize - 1) / kBlockSize : 0;
    for (int j = tid; j < dn; j += kCmpThreads) sm.dpage[j] = page_of(d0 / kBlockSize + j);
    moved = __reduce_min_sync(0xffffffffu, moved);
    if (lane == 0 && moved < kCmpSpan) atomicMin(&sm.moved, moved);
    __syncthreads();
    if (sm.moved < count) {
      auto go = [&](auto word, auto token_first) {
        move_span<decltype(word), decltype(token_first)::value, CLUSTER>(
            sl, sm, sm.moved, count, d0, rank, CLUSTER ? p.ctas : 1, p.dev_err);
      };
      if (slice < C::NK) {
        if constexpr (KVT == 16) go(uint4{}, False{});
        else go(uint2{}, False{});
      } else if (slice < C::NK + C::NV) {
        go(uint4{}, False{});
      } else if constexpr (G::I4) {
        if (slice < C::NK + C::NV + C::NS) go(uint16_t{}, True{});
        else if constexpr (VSVT == 16) go(uint4{}, False{});
        else go(uint16_t{}, False{});
      }
    }
    d0 += count;
  }
  if (slice == 0 && rank == 0 && tid == 0) p.new_lens[b] = d0;
  // no CTA of a cluster leaves while another may still wait at its barrier
  if constexpr (CLUSTER) cluster_sync_all();
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
cudaError_t compact_fmt(CompactParams p, int num_sms, cudaStream_t stream) {
  // Two CTAs fit an SM.  A slice gets one, or while that leaves half of the places free a
  // cluster of two, four or eight (a cluster of six measured slower than one of four: it
  // leaves SMs empty).
  int64_t slices = static_cast<int64_t>(p.batch) * CompactSlices<S, FMT, true>::N;
  p.ctas = 1;
  while (p.ctas < kCmpCluster && slices * p.ctas <= num_sms) p.ctas *= 2;
  const bool cluster = p.ctas > 1;
  if (!cluster) slices = static_cast<int64_t>(p.batch) * CompactSlices<S, FMT, false>::N;
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3(static_cast<unsigned>(slices * p.ctas));
  cfg.blockDim = dim3(kCmpThreads);
  cfg.dynamicSmemBytes = sizeof(CompactSmem);
  cfg.stream = stream;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = static_cast<unsigned>(p.ctas);
  attr[1].val.clusterDim.y = 1;
  attr[1].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = cluster ? 2 : 1;
  return cluster ? cudaLaunchKernelEx(&cfg, compact_kernel<S, FMT, true>, p)
                 : cudaLaunchKernelEx(&cfg, compact_kernel<S, FMT, false>, p);
}

template <class S>
cudaError_t prepare_pages() {
  auto set = [](auto kernel) {
    return cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                static_cast<int>(sizeof(CompactSmem)));
  };
  cudaError_t e = set(compact_kernel<S, RCP_PAGES_FP16, false>);
  if (e == cudaSuccess) e = set(compact_kernel<S, RCP_PAGES_FP8_E4M3, false>);
  if (e == cudaSuccess) e = set(compact_kernel<S, RCP_PAGES_INT4, false>);
  if (e == cudaSuccess) e = set(compact_kernel<S, RCP_PAGES_FP16, true>);
  if (e == cudaSuccess) e = set(compact_kernel<S, RCP_PAGES_FP8_E4M3, true>);
  if (e == cudaSuccess) e = set(compact_kernel<S, RCP_PAGES_INT4, true>);
  return e;
}

template <class S>
cudaError_t launch_compact(const CompactParams& p, int page_format, int num_sms,
                           cudaStream_t stream) {
  if (page_format == RCP_PAGES_FP8_E4M3)
    return compact_fmt<S, RCP_PAGES_FP8_E4M3>(p, num_sms, stream);
  if (page_format == RCP_PAGES_INT4) return compact_fmt<S, RCP_PAGES_INT4>(p, num_sms, stream);
  return compact_fmt<S, RCP_PAGES_FP16>(p, num_sms, stream);
}

template cudaError_t launch_copy_pages<ShapeMain>(const CopyParams&, const int32_t*, int, int,
                                                  cudaStream_t);
template cudaError_t launch_copy_pages<ShapeTiny>(const CopyParams&, const int32_t*, int, int,
                                                  cudaStream_t);
template cudaError_t prepare_pages<ShapeMain>();
template cudaError_t prepare_pages<ShapeTiny>();
template cudaError_t launch_compact<ShapeMain>(const CompactParams&, int, int, cudaStream_t);
template cudaError_t launch_compact<ShapeTiny>(const CompactParams&, int, int, cudaStream_t);

}  // namespace rcp
