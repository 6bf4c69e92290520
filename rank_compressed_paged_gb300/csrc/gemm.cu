// Tensor-core projections: the append's key / value projections (with, in the same
// launch, the decode's rank-space queries) and the chunked prefill's rank-space queries,
// as tcgen05 GEMMs D[128 x NT] = A[128 x K] * B[NT x K]^T.
//
// Both operands come from global memory through 2-D tensor maps with 128-byte swizzle
// (64 fp16 of K per row), four pipeline stages, one elected thread issuing
// tcgen05.mma.cta_group::1.kind::f16 into a TMEM accumulator.  When the token / query
// count is small, K is split over a thread-block cluster of KS CTAs; each CTA sends the
// rows owned by every peer to that peer's shared memory (distributed shared memory
// stores), a cluster barrier publishes them, and each CTA sums and writes its rows.
//
//   append, value job:  A = W_v rows [m0, m0+128) (K-major over H*d), B = v tokens,
//                       D[r][t] -> V page [slot_t / 16][slot_t % 16][m0 + r]
//   append, key job:    two heads h, h+1 at once as a block-diagonal product (K = 2d):
//                       A = [U_k,h 0; 0 U_k,h+1] (64-row boxes; the zero quadrants are
//                       boxes past the end of U_k, which the copy fills with zeros),
//                       B = k tokens of heads h and h+1 (adjacent columns),
//                       D[64 i + k][t] -> K page [slot_t / 16][h + i][slot_t % 16][k]
//   decode query job:   a key job with the decode queries as B (same launch as the
//                       append): D[64 i + k][q] = q~_{q,h+i,k}, stored fp32, scaled by
//                       log2(e)/sqrt(d), for the split-K scoring; a chunked prefill step
//                       puts its query projections (below) in the append's launch the
//                       same way.
//   query projection:   as a key job with the chunk's queries as B: D[k][q] = q~_{q,h,k},
//                       scaled by log2(e)/sqrt(d) and stored as an fp16 (hi, lo) pair
//                       (zero past r_k, up to 64), the prefill score MMA's A operand.
//   rotated key / query job (ROT kernels, rcp_rotary): U_k does not commute with the rotation of
//                       positions, so it comes first: the CTA waits for its whole tile of k (or
//                       q), rotates it in shared memory in fp32, and leaves it as an fp16
//                       (hi, lo) pair in place of the fp16 input, so that the product keeps
//                       fp32-level accuracy (one more MMA; the tensor pipe is idle here).
//                       Up to 192 tokens or queries; more: rotproj.cu.  An append of 37 tokens
//                       takes 7.6 us on E4M3 pages, a decode step's projections of 16 tokens and
//                       queries 10.2 from a cold cache (the factors' 9 MB set the pace).
#include <cuda.h>
#include <cuda_fp16.h>
#include <cuda_fp8.h>
#include <cuda_runtime.h>

#include <cstdint>

#include "launch.h"
#include "ptx.cuh"
#include "quant.cuh"
#include "rcp.h"
#include "shape.h"

namespace rcp {

constexpr int kGemmThreads = 128;
constexpr int kABytes = 128 * 64 * 2;   // one A stage: 128 rows x 64 K (or 64 K x 128 M)

enum GemmMode : int { kModeAppend = 0, kModeQproj = 2 };

template <int NT, int KS, int NB, int STG>
struct GemmSmem {
  static constexpr int B_BYTES = NT * 128;                     // one B operand stage
  static constexpr int STAGE = kABytes + NB * B_BYTES;
  // split-K receive buffer: KS partial slices of 128 / KS rows, rows RS floats apart (the
  // padding spreads the rows of a column over the banks)
  static constexpr int RS = NT + 4;
  static constexpr int RECV_OFF = STG * STAGE;
  static constexpr int RECV_BYTES = KS > 1 ? 128 * RS * 4 : 0;
  static constexpr int BAR_OFF = RECV_OFF + RECV_BYTES;        // full[S], empty[S], acc
  static constexpr int MISC_OFF = BAR_OFF + (2 * STG + 1) * 8;
  static constexpr int DST_OFF = MISC_OFF + 16;                // append: page offset per column
  static constexpr int RED_OFF = DST_OFF + NT * 8;             // 4-bit append: [4 warps][16]
  static constexpr int TOTAL = RED_OFF + 4 * 16 * 4;
  static constexpr int ALLOC = TOTAL + 1024;
  static constexpr int TMEM_COLS = NT < 32 ? 32 : NT;
  static_assert(STAGE % 1024 == 0, "stages must keep 1024-byte alignment");
  static_assert(MISC_OFF % 8 == 0 && DST_OFF % 8 == 0 && (RS * 4) % 16 == 0, "alignment");
  static_assert(ALLOC <= 227 * 1024, "shared memory budget");
};

struct GemmParams {
  // append
  const int64_t* slots;
  void* k_pages;
  void* v_pages;
  int32_t T;
  int32_t fmt;            // RCP_PAGES_*: fp16, E4M3 (round to nearest even, saturate) or
                          // 4-bit codes with per-group fp16 scales
  int64_t num_blocks;
  int32_t nq;             // decode queries (decode query jobs), prefill rows
  uint32_t* dev_err;
  // rank-space queries: chunked prefill fp16 hi / lo [nq][H][64]; decode fp32 [nq][H][r_k]
  void* qhi;
  void* qlo;
  float* qt;
  float qscale;
  // position rotation (ROT): rows [num_pos][rot_dim] of cosines, then sines; a null list of
  // positions leaves its operand as it is
  const float* rot_table;
  const int32_t* k_pos;
  const int32_t* q_pos;
  int32_t num_pos;
  int32_t rot_dim;
  int32_t interleaved;
  int32_t wait_at_exit;   // wait for the previous launch at exit (one CTA) instead of first
};

// Where one CTA's job reads and writes.
struct GemmJob {
  int kind;        // 0 value (append), 1 key (append), 3 prefill query, 4 decode query,
                   // -1 idle
  int a_x, a_y;    // tensor-map coordinates of A's first k-block (x innermost)
  int b_x, b_y;    // coordinates of B's first k-block
  int a_step_x, a_step_y, b_step_x;   // per-k-block coordinate steps
  int kb0, kb1;    // k-block range of this CTA
  int m0;          // first output row (value rank row) / head index
  int n0;          // first token / query of the tile
  bool reduce;     // cluster split-K reduction
};

template <class S, int MODE, int NT, int KS>
__device__ __forceinline__ GemmJob gemm_job(uint32_t rank, int T, bool prefill_q) {
  GemmJob j{};
  const int cluster = blockIdx.x / KS;
  if constexpr (MODE == kModeAppend) {
    constexpr int NM = (S::R + 127) / 128;
    constexpr int NP = S::H / 2;                 // head pairs
    constexpr int NKG = (NP + KS - 1) / KS;
    constexpr int KBV = S::H * S::D / 64;
    constexpr int KBK = S::D / 64;
    // the append's clusters come first (the value jobs of every token tile, then their key
    // jobs), then the query jobs (head pairs, per query tile): decode or prefill queries
    const int app_clusters = (T + NT - 1) / NT * (NM + NKG);
    if (cluster >= app_clusters) {
      const int qc = cluster - app_clusters;
      const int pr = (qc % NKG) * KS + static_cast<int>(rank);
      j.kind = pr < NP ? (prefill_q ? 3 : 4) : -1;
      j.m0 = 2 * pr;
      j.n0 = (qc / NKG) * NT;
      j.kb0 = 0;
      j.kb1 = 2 * KBK;
      j.a_x = 0; j.a_y = j.m0 * S::RK; j.a_step_x = 64; j.a_step_y = 0;
      j.b_x = j.m0 * S::D; j.b_y = j.n0; j.b_step_x = 64;
      j.reduce = false;
      return j;
    }
    // value jobs of every token tile first (K = H d: the long ones, so they all start in
    // the first wave), then the key jobs
    const int ntile = (T + NT - 1) / NT;
    const bool value_job = cluster < ntile * NM;
    const int tile = value_job ? cluster / NM : (cluster - ntile * NM) / NKG;
    const int sub = value_job ? cluster % NM : NM + (cluster - ntile * NM) % NKG;
    j.n0 = tile * NT;
    if (sub < NM) {
      j.kind = 0;
      j.m0 = sub * 128;
      j.kb0 = static_cast<int>(rank) * KBV / KS;
      j.kb1 = (static_cast<int>(rank) + 1) * KBV / KS;
      j.a_x = j.kb0 * 64; j.a_y = j.m0; j.a_step_x = 64; j.a_step_y = 0;
      j.b_x = j.kb0 * 64; j.b_y = j.n0; j.b_step_x = 64;
      j.reduce = KS > 1;
    } else {
      const int pr = (sub - NM) * KS + static_cast<int>(rank);
      j.kind = pr < NP ? 1 : -1;
      j.m0 = 2 * pr;                             // first head of the pair
      j.kb0 = 0;
      j.kb1 = 2 * KBK;
      j.a_x = 0; j.a_y = j.m0 * S::RK; j.a_step_x = 64; j.a_step_y = 0;
      j.b_x = j.m0 * S::D; j.b_y = j.n0; j.b_step_x = 64;
      j.reduce = false;
    }
  } else if constexpr (MODE == kModeQproj) {
    // two heads h, h+1 at once, block-diagonal over K = 2d as the append's key jobs
    const int pr = blockIdx.x % (S::H / 2);
    j.kind = 3;
    j.m0 = 2 * pr;
    j.n0 = (blockIdx.x / (S::H / 2)) * NT;
    j.kb0 = 0;
    j.kb1 = 2 * (S::D / 64);
    j.a_x = 0; j.a_y = j.m0 * S::RK; j.a_step_x = 64; j.a_step_y = 0;
    j.b_x = j.m0 * S::D; j.b_y = j.n0; j.b_step_x = 64;
    j.reduce = false;
  }
  return j;
}

// Page offset (in fp16 elements; 4-bit pages: the slot itself) that column col of an append
// job writes from, or -1 when the token is padding (slot < 0), past the token count, or has
// an out-of-range slot (which also raises the device error bit).  Computed once per column
// before the epilogue so that the store loop issues no dependent loads.
template <class S>
__device__ __forceinline__ int64_t append_dst(const GemmParams& p, const GemmJob& j, int col) {
  const int n = j.n0 + col;
  if ((j.kind != 0 && j.kind != 1) || n >= p.T) return -1;
  const int64_t s = p.slots[n];
  if (s < 0) return -1;
  if (s >= p.num_blocks * kBlockSize) {
    atomicOr(p.dev_err, RCP_DEVERR_BAD_SLOT);
    return -1;
  }
  if (p.k_pos != nullptr && static_cast<uint32_t>(p.k_pos[n]) >= static_cast<uint32_t>(p.num_pos)) {
    atomicOr(p.dev_err, RCP_DEVERR_BAD_POS);
    return -1;
  }
  if (p.fmt == RCP_PAGES_INT4) return s;
  const int64_t blk = s / kBlockSize, off = s % kBlockSize;
  return j.kind == 0 ? (blk * kBlockSize + off) * S::R
                     : ((blk * S::H + j.m0) * kBlockSize + off) * S::RK;
}

// 4-bit pages: quantize NC finished columns c0 .. c0+NC-1 of an append job, held by every
// thread as v[] for its row (TMEM lane), and store codes and scales.  A group is 64 rows:
// a key row of one head (rows 0..63, 64..127 of a key-pair job; rows at or past r_k of a
// head are not coefficients) or 64 value coefficients (m0 + 0..63, m0 + 64..127).  Per
// group: the smallest fp16 scale with 7 * scale >= max |x|, codes x / scale rounded to
// nearest, ties to even, in [-7, 7]; two codes per byte, the even row in the low nibble.
// All kGemmThreads threads take part (block barriers).
template <class S, int NC>
__device__ __forceinline__ void int4_store_columns(const GemmParams& p, const GemmJob& j,
                                                   const int64_t* dst, float* red, int c0,
                                                   const float* v) {
  using P = Int4Page<S>;
  const int row = threadIdx.x, warp = row >> 5, lane = row & 31;
  const bool valid = j.kind == 1 ? (row & 63) < S::RK : j.m0 + row < S::R;
  float a[NC];
#pragma unroll
  for (int e = 0; e < NC; ++e) {
    a[e] = valid ? fabsf(v[e]) : 0.f;
#pragma unroll
    for (int o = 16; o >= 1; o >>= 1) a[e] = fmaxf(a[e], __shfl_xor_sync(0xffffffffu, a[e], o));
  }
  if (lane == 0)
#pragma unroll
    for (int e = 0; e < NC; ++e) red[warp * 16 + e] = a[e];
  __syncthreads();
  // every column's scale and code first (independent chains), then the stores
  __half shs[NC];
  int codes[NC];
#pragma unroll
  for (int e = 0; e < NC; ++e) {
    const float amax = fmaxf(red[warp * 16 + e], red[(warp ^ 1) * 16 + e]);
    const __half sh = int4_scale(amax);
    shs[e] = sh;
    const float sf = __half2float(sh);
    codes[e] = (valid && sf > 0.f) ? max(-7, min(7, rne_div(v[e], sf, __fdividef(1.f, sf)))) : 0;
  }
#pragma unroll
  for (int e = 0; e < NC; ++e) {
    const __half sh = shs[e];
    const int code = codes[e];
    const int hi = __shfl_down_sync(0xffffffffu, code, 1);   // the next row's code
    const int64_t s = dst[c0 + e];
    if (s < 0 || !valid) continue;
    const int64_t blk = s / kBlockSize, off = s % kBlockSize;
    uint8_t* page;
    int64_t cbyte, sidx;
    bool first;   // the group's first row stores its scale
    if (j.kind == 1) {
      const int hh = j.m0 + (row >> 6), rr = row & 63;
      page = static_cast<uint8_t*>(p.k_pages) + blk * P::KBYTES;
      cbyte = ((hh * kBlockSize + off) * S::RK + rr) / 2;
      sidx = hh * kBlockSize + off;
      first = rr == 0;
      if (first) reinterpret_cast<__half*>(page + P::KCODES)[sidx] = sh;
    } else {
      const int r = j.m0 + row;
      page = static_cast<uint8_t*>(p.v_pages) + blk * P::VBYTES;
      cbyte = (off * S::R + r) / 2;
      sidx = off * (S::R / 64) + r / 64;
      first = (r & 63) == 0;
      if (first) reinterpret_cast<__half*>(page + P::VCODES)[sidx] = sh;
    }
    if ((row & 1) == 0) page[cbyte] = static_cast<uint8_t>((code & 0xF) | ((hi & 0xF) << 4));
  }
  __syncthreads();   // red[] is reused by the next call
}

// Write one finished output element (row, column) of a job.
template <class S>
__device__ __forceinline__ void gemm_store(const GemmParams& p, const GemmJob& j,
                                           const int64_t* dst, int row, int col, float v) {
  const int n = j.n0 + col;
  if (j.kind == 4) {
    // decode query: rows 0..63 are head m0's ranks, rows 64..127 head m0 + 1's
    const int hh = row >> 6, rr = row & 63;
    if (rr < S::RK && n < p.nq)
      p.qt[(static_cast<size_t>(n) * S::H + j.m0 + hh) * S::RK + rr] = v * p.qscale;
    return;
  }
  if (j.kind == 3) {
    // rows 0..63 are head m0's ranks, rows 64..127 head m0 + 1's; rows past r_k hold the
    // next heads' products and are written as the zero padding up to 64
    const int hh = row >> 6, rr = row & 63;
    if (n >= p.nq) return;
    const size_t at = (static_cast<size_t>(n) * S::H + j.m0 + hh) * 64 + rr;
    float q = rr < S::RK ? v * p.qscale : 0.f;
    const __half hi = __float2half_rn(q);
    static_cast<__half*>(p.qhi)[at] = hi;
    static_cast<__half*>(p.qlo)[at] = __float2half_rn(q - __half2float(hi));
    return;
  }
  const int64_t d = dst[col];
  if (d < 0) return;
  int64_t at;
  void* pages;
  if (j.kind == 0) {
    const int r = j.m0 + row;
    if (r >= S::R) return;
    at = d + r;
    pages = p.v_pages;
  } else {
    // rows 0..63 belong to head m0, rows 64..127 to head m0 + 1 (next head in the page)
    const int hh = row >> 6, rr = row & 63;
    if (rr >= S::RK) return;
    at = d + hh * kBlockSize * S::RK + rr;
    pages = p.k_pages;
  }
  if (p.fmt == RCP_PAGES_FP8_E4M3)
    static_cast<__nv_fp8_storage_t*>(pages)[at] = __nv_cvt_float_to_fp8(v, __NV_SATFINITE, __NV_E4M3);
  else
    static_cast<__half*>(pages)[at] = __float2half_rn(v);
}

// One warp's epilogue staging area: 16 columns x 32 rows of at most 4 bytes (fp32 decode
// queries; the prefill queries' fp16 hi and lo parts take two 1 KB planes).
constexpr int kEpiWarpBytes = 16 * 32 * 4;

// Write columns c0 .. c0+15 of a job's tile for rows 32 warp .. 32 warp + 31 (v[] holds this
// lane's row).  In every destination a column's rows are contiguous (a page row's value
// coefficients, a head's ranks), so the warp transposes the block through its staging area
// and writes each column's run of rows as 16-byte pieces rather than an element per lane.
// ES: bytes per element (4 decode queries, 2 fp16 pages and prefill queries, 1 E4M3 pages);
// PL: planes (2 for the prefill queries' hi and lo parts).  Both fixed at compile time, so
// that the piece loop unrolls with shifts and masks for its indexes.
template <class S, int ES, int PL>
__device__ __forceinline__ void gemm_store_block(const GemmParams& p, const GemmJob& j,
                                                 const int64_t* dst, uint8_t* stage, int warp,
                                                 int lane, int c0, const float (&v)[16]) {
  static_assert(S::R % 32 == 0 && S::RK % 16 == 0, "runs of whole 16-byte pieces");
  constexpr int NCH = 32 * ES / 16;    // 16-byte pieces of a column's 32 rows, per plane
  constexpr int PER = 16 * NCH;        // pieces of the block, per plane
  static_assert((PL * PER) % 32 == 0 && PL * 16 * 32 * ES <= kEpiWarpBytes, "staging");
  const int hh = warp >> 1;            // key / query jobs: head m0 + hh
  const int rr0 = (warp & 1) * 32;     // ... ranks rr0 .. rr0 + 31
  int nvalid;
  if constexpr (ES == 4) {             // decode queries, fp32
    nvalid = min(32, max(0, S::RK - rr0));
    float* s = reinterpret_cast<float*>(stage);
#pragma unroll
    for (int e = 0; e < 16; ++e) s[e * 32 + lane] = v[e] * p.qscale;
  } else if constexpr (PL == 2) {      // prefill queries, fp16 hi and lo
    // ranks past r_k hold the next heads' products and are written as zero padding
    nvalid = 32;
    __half* s = reinterpret_cast<__half*>(stage);
    const bool rank = rr0 + lane < S::RK;
#pragma unroll
    for (int e = 0; e < 16; ++e) {
      const float q = rank ? v[e] * p.qscale : 0.f;
      const __half hi = __float2half_rn(q);
      s[e * 32 + lane] = hi;
      s[512 + e * 32 + lane] = __float2half_rn(q - __half2float(hi));
    }
  } else {                             // append: value or key page coefficients
    nvalid = j.kind == 0 ? min(32, max(0, S::R - (j.m0 + warp * 32)))
                         : min(32, max(0, S::RK - rr0));
    if constexpr (ES == 1) {
#pragma unroll
      for (int e = 0; e < 16; ++e)
        stage[e * 32 + lane] = __nv_cvt_float_to_fp8(v[e], __NV_SATFINITE, __NV_E4M3);
    } else {
      __half* s = reinterpret_cast<__half*>(stage);
#pragma unroll
      for (int e = 0; e < 16; ++e) s[e * 32 + lane] = __float2half_rn(v[e]);
    }
  }
  __syncwarp();
  const int nvc = nvalid * ES / 16;    // pieces of a column that hold valid rows
#pragma unroll
  for (int it = 0; it < PL * PER / 32; ++it) {
    const int i = lane + 32 * it;
    const int plane = i / PER, c = (i % PER) / NCH, k = i % NCH;
    if (k >= nvc) continue;
    uint8_t* out;
    if constexpr (ES == 4 || PL == 2) {
      const int n = j.n0 + c0 + c;
      if (n >= p.nq) continue;
      const size_t hrow = static_cast<size_t>(n) * S::H + j.m0 + hh;
      if constexpr (ES == 4)
        out = reinterpret_cast<uint8_t*>(p.qt) + (hrow * S::RK + rr0) * 4;
      else
        out = static_cast<uint8_t*>(plane ? p.qlo : p.qhi) + (hrow * 64 + rr0) * 2;
    } else {
      const int64_t d = dst[c0 + c];
      if (d < 0) continue;
      out = j.kind == 0
                ? static_cast<uint8_t*>(p.v_pages) + (d + j.m0 + warp * 32) * ES
                : static_cast<uint8_t*>(p.k_pages) + (d + hh * kBlockSize * S::RK + rr0) * ES;
    }
    *reinterpret_cast<uint4*>(out + k * 16) =
        *reinterpret_cast<const uint4*>(stage + plane * 1024 + c * 32 * ES + k * 16);
  }
  __syncwarp();   // the staging area is rewritten by the next block
}

// Shared memory of a rotated job: the k-blocks of A, then of B hi, then of B lo.
template <class S, int NT>
struct RotSmem {
  static constexpr int NKB = 2 * (S::D / 64);            // k-blocks: both heads'
  static constexpr int B_BYTES = NT * 128;
  static constexpr int HI_OFF = NKB * kABytes;
  static constexpr int LO_OFF = HI_OFF + NKB * B_BYTES;
  static constexpr int END = LO_OFF + NKB * B_BYTES;
};

// Rotates the rows n0 .. n0 + NT - 1 (below n) of the two heads in B hi, in place, and leaves
// what their fp16 rounding drops in B lo.  A unit is a 16-byte chunk (eight elements) of a row
// with its partners' chunk; both heads of a row take the same angles.  wait(): the rows have
// landed (called once the first unit's angles are on their way).
template <class S, int NT, class Wait>
__device__ __forceinline__ bool rotate_rows(const GemmParams& p, uint8_t* sm, int n0, int n,
                                            const int32_t* pos, bool query, Wait wait) {
  using L = RotSmem<S, NT>;
  constexpr int CH = S::D / 8, KBK = S::D / 64;
  const int half = p.rot_dim / 2, hc = half / 8;         // pairs, and chunks of their first elements
  const bool inter = p.interleaved != 0;
  // half-split pairs: units 0 .. hc-1 rotate chunks (u, u + hc), the rest keep chunk u + hc;
  // interleaved: unit u is chunk u, rotated below 2 hc
  const int units = inter ? CH : CH - hc, nrot = inter ? 2 * hc : hc;
  auto chunk = [&](int hh, int row, int c) {             // byte offset among an operand's k-blocks
    return (hh * KBK + (c >> 3)) * L::B_BYTES + row * 128 + (((c & 7) ^ (row & 7)) << 4);
  };
  uint8_t* hi = sm + L::HI_OFF;
  uint8_t* lo = sm + L::LO_OFF;
  // kBatch units at a time: their angles, from L2, are all on the way before the first is used
  // (one at a time: 64 tokens 12.4 us instead of 7.6)
  constexpr int kBatch = 4;
  const int items = min(NT, n - n0) * units;
  bool ok = true;
  for (int it0 = 0; it0 == 0 || it0 < items; it0 += kBatch * kGemmThreads) {
    int rows[kBatch], us[kBatch];
    uint32_t ats[kBatch];
    float4 ang[kBatch][4];   // of the unit's pairs: cosines, sines (eight each, or four interleaved)
#pragma unroll
    for (int k = 0; k < kBatch; ++k) {
      const int it = it0 + k * kGemmThreads + threadIdx.x;
      rows[k] = it < items ? it / units : -1;
      us[k] = it - rows[k] * units;
      ats[k] = rows[k] >= 0 ? static_cast<uint32_t>(pos[n0 + rows[k]]) : 0xFFFFFFFFu;
    }
#pragma unroll
    for (int k = 0; k < kBatch; ++k) {
      if (ats[k] >= static_cast<uint32_t>(p.num_pos) || us[k] >= nrot) continue;
      const float4* t = reinterpret_cast<const float4*>(
          p.rot_table + static_cast<int64_t>(ats[k]) * p.rot_dim + us[k] * (inter ? 4 : 8));
      ang[k][0] = __ldg(t);
      ang[k][2] = __ldg(t + half / 4);
      if (!inter) {
        ang[k][1] = __ldg(t + 1);
        ang[k][3] = __ldg(t + half / 4 + 1);
      }
    }
    if (it0 == 0) ok = wait();
    if (!ok) break;
#pragma unroll
    for (int k = 0; k < kBatch; ++k) {
      const int row = rows[k], u = us[k];
      if (row < 0) continue;
      const bool in = ats[k] < static_cast<uint32_t>(p.num_pos);
      if (!in && query) {
        // a query without a position counts as zero (a key without one is not stored)
        if (u == 0) atomicOr(p.dev_err, RCP_DEVERR_BAD_POS);
        for (int hh = 0; hh < 2; ++hh)
          for (int c = u; c < CH; c += units) {
            *reinterpret_cast<uint4*>(hi + chunk(hh, row, c)) = make_uint4(0, 0, 0, 0);
            *reinterpret_cast<uint4*>(lo + chunk(hh, row, c)) = make_uint4(0, 0, 0, 0);
          }
        continue;
      }
      if (!in) continue;
      if (u >= nrot) {
        const int c = inter ? u : u + hc;
        for (int hh = 0; hh < 2; ++hh)
          *reinterpret_cast<uint4*>(lo + chunk(hh, row, c)) = make_uint4(0, 0, 0, 0);
        continue;
      }
      const float4 ca = ang[k][0], cb = ang[k][1], sa = ang[k][2], sb = ang[k][3];
      const float cs[8] = {ca.x, ca.y, ca.z, ca.w, cb.x, cb.y, cb.z, cb.w};
      const float sn[8] = {sa.x, sa.y, sa.z, sa.w, sb.x, sb.y, sb.z, sb.w};
#pragma unroll
      for (int hh = 0; hh < 2; ++hh) {
        if (inter) {
          const int o = chunk(hh, row, u);
          const uint4 x = *reinterpret_cast<const uint4*>(hi + o);
          const uint32_t xw[4] = {x.x, x.y, x.z, x.w};
          uint32_t h[4], l[4];
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&xw[j]));
            split_pair(fmaf(f.x, cs[j], -(f.y * sn[j])), fmaf(f.y, cs[j], f.x * sn[j]), h[j], l[j]);
          }
          *reinterpret_cast<uint4*>(hi + o) = make_uint4(h[0], h[1], h[2], h[3]);
          *reinterpret_cast<uint4*>(lo + o) = make_uint4(l[0], l[1], l[2], l[3]);
        } else {
          const int o1 = chunk(hh, row, u), o2 = chunk(hh, row, u + hc);
          const uint4 x1 = *reinterpret_cast<const uint4*>(hi + o1);
          const uint4 x2 = *reinterpret_cast<const uint4*>(hi + o2);
          const uint32_t w1[4] = {x1.x, x1.y, x1.z, x1.w}, w2[4] = {x2.x, x2.y, x2.z, x2.w};
          uint32_t h1[4], l1[4], h2[4], l2[4];
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            const float2 a = __half22float2(*reinterpret_cast<const __half2*>(&w1[j]));
            const float2 b = __half22float2(*reinterpret_cast<const __half2*>(&w2[j]));
            const float c0 = cs[2 * j], c1 = cs[2 * j + 1], s0 = sn[2 * j], s1 = sn[2 * j + 1];
            split_pair(fmaf(a.x, c0, -(b.x * s0)), fmaf(a.y, c1, -(b.y * s1)), h1[j], l1[j]);
            split_pair(fmaf(b.x, c0, a.x * s0), fmaf(b.y, c1, a.y * s1), h2[j], l2[j]);
          }
          *reinterpret_cast<uint4*>(hi + o1) = make_uint4(h1[0], h1[1], h1[2], h1[3]);
          *reinterpret_cast<uint4*>(hi + o2) = make_uint4(h2[0], h2[1], h2[2], h2[3]);
          *reinterpret_cast<uint4*>(lo + o1) = make_uint4(l1[0], l1[1], l1[2], l1[3]);
          *reinterpret_cast<uint4*>(lo + o2) = make_uint4(l2[0], l2[1], l2[2], l2[3]);
        }
      }
    }
  }
  return ok;
}

template <class S, int MODE, int NT, int KS, int STG, bool ROT = false>
__global__ void __launch_bounds__(kGemmThreads, 1)
    gemm_kernel(const __grid_constant__ CUtensorMap map_a, const __grid_constant__ CUtensorMap map_a2,
                const __grid_constant__ CUtensorMap map_b, const __grid_constant__ CUtensorMap map_b2,
                const __grid_constant__ CUtensorMap map_b3, const GemmParams p) {
  constexpr int kGemmStages = STG;
  using L = GemmSmem<NT, KS, 1, STG>;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* sm = reinterpret_cast<uint8_t*>(
      (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~static_cast<uintptr_t>(1023));
  uint64_t* full = reinterpret_cast<uint64_t*>(sm + L::BAR_OFF);
  uint64_t* empty = full + kGemmStages;
  uint64_t* accb = empty + kGemmStages;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(sm + L::MISC_OFF);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(sm + L::MISC_OFF + 4);
  float* recv = reinterpret_cast<float*>(sm + L::RECV_OFF);

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const uint32_t rank = KS > 1 ? cluster_ctarank() : 0;
  using RL = RotSmem<S, NT>;
  static_assert(!ROT || (MODE == kModeAppend && RL::END <= STG * L::STAGE && RL::NKB <= STG), "rotated jobs");
  const GemmJob j = gemm_job<S, MODE, NT, KS>(rank, p.T, p.qhi != nullptr);
  // value jobs read W_v through map_a and their tokens through map_b;
  // key jobs (and the query jobs of the query-projection launch) read U_k through map_a2
  // and their rows through map_b2; query jobs of an append launch read U_k through map_a2
  // and the queries through map_b3
  const bool uk = j.kind == 1 || j.kind == 3 || j.kind == 4;
  const bool qjob = j.kind == 4 || (MODE == kModeAppend && j.kind == 3);
  const CUtensorMap* amap = uk ? &map_a2 : &map_a;
  const CUtensorMap* bmap = qjob ? &map_b3 : (uk ? &map_b2 : &map_b);
  const bool rot = ROT && uk;   // uniform over the CTA

  if (threadIdx.x == 0) {
    for (int s = 0; s < kGemmStages; ++s) {
      mbar_init(&full[s], 1);
      mbar_init(&empty[s], 1);
    }
    mbar_init(accb, 1);
    *abort_flag = 0;
    fence_mbar_init();
  }
  if (warp == 1) {
    tmem_alloc(tmem_slot, L::TMEM_COLS);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;
  if (j.reduce) cluster_sync_all();   // every peer is running before any remote store

  const int nkb = j.kind >= 0 ? j.kb1 - j.kb0 : 0;
  auto load_a = [&](int kb, int s) {
    uint8_t* st = sm + s * (rot ? kABytes : L::STAGE);
    if ((MODE == kModeAppend && (j.kind == 1 || j.kind == 3 || j.kind == 4)) ||
        MODE == kModeQproj) {
      // block-diagonal pair: k-blocks [0, d/64) meet head m0's rows (top), the rest head
      // m0 + 1's (bottom); the other half is a box past the last row of U_k (zeros)
      constexpr int KBK = S::D / 64, OOB = S::H * S::RK;
      const int half = kb / KBK, kk = kb % KBK;
      tma_load_2d(st, amap, kk * 64, half == 0 ? j.m0 * S::RK : OOB, &full[s]);
      tma_load_2d(st + kABytes / 2, amap, kk * 64, half == 1 ? (j.m0 + 1) * S::RK : OOB, &full[s]);
    } else {
      tma_load_2d(st, amap, j.a_x + kb * j.a_step_x, j.a_y, &full[s]);
    }
  };
  auto load_b = [&](int kb, int s) {
    uint8_t* st = rot ? sm + RL::HI_OFF + s * RL::B_BYTES : sm + s * L::STAGE + kABytes;
    tma_load_2d(st, bmap, j.b_x + kb * j.b_step_x, j.b_y, &full[s]);
  };
  // A is always a factor (W_v or U_k), which no kernel writes: its first stages are
  // fetched before waiting on the previous kernel, whose outputs only B may read.
  const uint32_t kStageTx = kABytes + (rot ? RL::B_BYTES : L::B_BYTES);
  const int pre = nkb < kGemmStages ? nkb : kGemmStages;
  if (warp == 0 && lane == 0 && nkb > 0) {
    prefetch_tmap(amap);
    prefetch_tmap(bmap);
    for (int kb = 0; kb < pre; ++kb) {
      mbar_arrive_expect_tx(&full[kb], kStageTx);
      load_a(kb, kb);
    }
  }
  // operands written by the previous kernel are visible (unless that kernel writes nothing
  // this one touches: then it is waited for at exit, so that kernels after this one still
  // see its results)
  if (!p.wait_at_exit) griddep_wait();
  griddep_launch();

  if (rot) {
    // ------------------------------------------ rotated job: the whole tile, step by step
    if constexpr (ROT) {
      if (warp == 0 && lane == 0)
        for (int kb = 0; kb < nkb; ++kb) load_b(kb, kb);
      __syncwarp();
      const int32_t* pos = qjob ? p.q_pos : p.k_pos;
      auto landed = [&]() {
        bool all = true;
        for (int kb = 0; kb < nkb; ++kb) all = mbar_wait(&full[kb], 0, abort_flag, p.dev_err) && all;
        return all;
      };
      const bool ok = __syncthreads_and(
          pos ? rotate_rows<S, NT>(p, sm, j.n0, qjob ? p.nq : p.T, pos, qjob, landed) : landed());
      if (pos) fence_proxy_async_smem();   // generic stores -> the MMAs' async-proxy reads
      __syncthreads();
      if (warp == 1 && lane == 0) {
        constexpr uint32_t idesc = make_idesc_f16(128, NT, false, false);
        tc_fence_after();
        for (int kb = 0; ok && kb < nkb; ++kb) {
          const uint32_t a0 = smem_u32(sm + kb * kABytes);
          const uint32_t b0 = smem_u32(sm + RL::HI_OFF + kb * RL::B_BYTES);
          const uint32_t b1 = smem_u32(sm + RL::LO_OFF + kb * RL::B_BYTES);
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            const uint64_t ad = make_sdesc(a0 + k * 32, 16, 1024, kSwizzle128B);
            umma_f16(tmem, ad, make_sdesc(b0 + k * 32, 16, 1024, kSwizzle128B), idesc,
                     (kb > 0 || k > 0) ? 1u : 0u);
            if (pos) umma_f16(tmem, ad, make_sdesc(b1 + k * 32, 16, 1024, kSwizzle128B), idesc, 1u);
          }
        }
        umma_commit(accb);
        if (!ok) {
          mbar_wait_drain(accb, 0);
          for (int kb = 0; kb < nkb; ++kb) mbar_wait_drain(&full[kb], 0);
        }
      }
    }
  } else if (warp == 0 && lane == 0 && nkb > 0) {
    // -------------------------------------------------------------- TMA producer
    int issued = 0;
    for (int kb = 0; kb < nkb; ++kb) {
      const int s = kb % kGemmStages;
      if (kb >= pre) {
        if (!mbar_wait(&empty[s], ((kb / kGemmStages) - 1) & 1, abort_flag, p.dev_err)) break;
        mbar_arrive_expect_tx(&full[s], kStageTx);
        load_a(kb, s);
      }
      load_b(kb, s);
      ++issued;
    }
    if (*abort_flag)
      for (int i = (issued > kGemmStages ? issued - kGemmStages : 0); i < issued; ++i)
        mbar_wait_drain(&full[i % kGemmStages], (i / kGemmStages) & 1);
  } else if (warp == 1 && lane == 0 && nkb > 0) {
    // -------------------------------------------------------------- MMA issuer
    constexpr uint32_t idesc = make_idesc_f16(128, NT, false, false);
    int kb = 0;
    for (; kb < nkb; ++kb) {
      const int s = kb % kGemmStages;
      if (!mbar_wait(&full[s], (kb / kGemmStages) & 1, abort_flag, p.dev_err)) break;
      tc_fence_after();
      const uint32_t a0 = smem_u32(sm + s * L::STAGE);
      const uint32_t b0 = a0 + kABytes;
#pragma unroll
      for (int k = 0; k < 4; ++k) {   // four K=16 steps per 64-wide k-block
        const uint64_t ad = make_sdesc(a0 + k * 32, 16, 1024, kSwizzle128B);
        const uint64_t bd = make_sdesc(b0 + k * 32, 16, 1024, kSwizzle128B);
        umma_f16(tmem, ad, bd, idesc, (kb > 0 || k > 0) ? 1u : 0u);
      }
      umma_commit(&empty[s]);
    }
    umma_commit(accb);
    if (kb < nkb) mbar_wait_drain(accb, 0);
  }
  __syncwarp();
  int64_t* dst_s = reinterpret_cast<int64_t*>(sm + L::DST_OFF);
  if (MODE == kModeAppend) {
    // idle warps get here while the main loop runs; the two issuing lanes join after it
    for (int c = threadIdx.x; c < NT; c += kGemmThreads) dst_s[c] = append_dst<S>(p, j, c);
    __syncthreads();
  }

  // ------------------------------------------------------------------ epilogue
  // warp-uniform, since TMEM loads are warp-collective
  const bool have_acc = __all_sync(0xffffffffu, nkb > 0 && mbar_wait(accb, 0, abort_flag, p.dev_err));
  tc_fence_after();
  const int row = warp * 32 + lane;                          // TMEM lane = output row
  const uint32_t trow = tmem + (static_cast<uint32_t>(warp * 32) << 16);
  // 4-bit pages: an append job quantizes whole 64-row groups (uniform over the CTA, and
  // over the cluster for split-K value jobs)
  const bool int4 = MODE == kModeAppend && p.fmt == RCP_PAGES_INT4 && (j.kind == 0 || j.kind == 1);
  float* red = reinterpret_cast<float*>(sm + L::RED_OFF);
  if (int4 && !j.reduce) {
#pragma unroll 1
    for (int c0 = 0; c0 < NT; c0 += 16) {
      float v[16];
      if (have_acc) {
        tmem_ld16(trow + c0, v);
        tmem_wait_ld();
      } else {
#pragma unroll
        for (int e = 0; e < 16; ++e) v[e] = 0.f;
      }
      int4_store_columns<S, 16>(p, j, dst_s, red, c0, v);
    }
  } else if (int4) {
    if constexpr (KS > 1) {
    // split-K: column c belongs to peer c / CPC, which receives every row of it (a group
    // spans 64 rows) in slot [my rank][row][c % CPC]
    constexpr int CPC = NT / KS;
    static_assert(CPC >= 1 && CPC <= 16 && NT % KS == 0, "4-bit split-K columns");
    const uint32_t recv_local = smem_u32(recv);
#pragma unroll 1
    for (int c0 = 0; c0 < NT; c0 += 16) {
      float v[16];
      if (have_acc) {
        tmem_ld16(trow + c0, v);
        tmem_wait_ld();
      } else {
#pragma unroll
        for (int e = 0; e < 16; ++e) v[e] = 0.f;
      }
      if constexpr (CPC % 4 == 0) {   // four columns of one peer per 16-byte store
#pragma unroll
        for (int e = 0; e < 16; e += 4) {
          const int col = c0 + e;
          st_cluster_v4(map_to_rank(recv_local, static_cast<uint32_t>(col / CPC)) +
                            ((rank * 128 + row) * CPC + col % CPC) * 4,
                        v[e], v[e + 1], v[e + 2], v[e + 3]);
        }
      } else {
#pragma unroll
        for (int e = 0; e < 16; ++e) {
          const int col = c0 + e;
          st_cluster_f32(map_to_rank(recv_local, static_cast<uint32_t>(col / CPC)) +
                             ((rank * 128 + row) * CPC + col % CPC) * 4,
                         v[e]);
        }
      }
    }
    cluster_sync_all();
    float v[CPC];
#pragma unroll
    for (int c = 0; c < CPC; ++c) {
      float acc = 0.f;
#pragma unroll
      for (int s = 0; s < KS; ++s) acc += recv[(s * 128 + row) * CPC + c];
      v[c] = acc;
    }
    int4_store_columns<S, CPC>(p, j, dst_s, red, static_cast<int>(rank) * CPC, v);
    }
  } else if (!j.reduce) {
    if (have_acc) {
      // the pipeline stages are idle once the accumulator is complete: each warp stages its
      // blocks in the first stage
      static_assert(4 * kEpiWarpBytes <= L::STAGE, "epilogue staging fits in one stage");
      uint8_t* stage = sm + warp * kEpiWarpBytes;
      auto blocks = [&](auto store) {
#pragma unroll 1
        for (int c0 = 0; c0 < NT; c0 += 16) {
          float v[16];
          tmem_ld16(trow + c0, v);
          tmem_wait_ld();
          store(c0, v);
        }
      };
      if (j.kind == 4)
        blocks([&](int c0, const float(&v)[16]) { gemm_store_block<S, 4, 1>(p, j, dst_s, stage, warp, lane, c0, v); });
      else if (j.kind == 3)
        blocks([&](int c0, const float(&v)[16]) { gemm_store_block<S, 2, 2>(p, j, dst_s, stage, warp, lane, c0, v); });
      else if (p.fmt == RCP_PAGES_FP8_E4M3)
        blocks([&](int c0, const float(&v)[16]) { gemm_store_block<S, 1, 1>(p, j, dst_s, stage, warp, lane, c0, v); });
      else
        blocks([&](int c0, const float(&v)[16]) { gemm_store_block<S, 2, 1>(p, j, dst_s, stage, warp, lane, c0, v); });
    }
  } else {
    // split-K: row r belongs to peer r / RPC; send it to slot [my rank] of that peer
    constexpr int RPC = 128 / KS;
    const uint32_t recv_local = smem_u32(recv);
    const uint32_t dst_rank = static_cast<uint32_t>(row / RPC);
    const uint32_t dst = map_to_rank(recv_local, dst_rank) +
                         ((rank * RPC + (row % RPC)) * L::RS) * 4;
#pragma unroll 1
    for (int c0 = 0; c0 < NT; c0 += 16) {
      float v[16];
      if (have_acc) {
        tmem_ld16(trow + c0, v);
        tmem_wait_ld();
      } else {
#pragma unroll
        for (int e = 0; e < 16; ++e) v[e] = 0.f;
      }
#pragma unroll
      for (int e = 0; e < 16; e += 4)
        st_cluster_v4(dst + (c0 + e) * 4, v[e], v[e + 1], v[e + 2], v[e + 3]);
    }
    cluster_sync_all();
    // sum the KS partial slices of my RPC rows and write them
    for (int i = threadIdx.x; i < RPC * NT; i += kGemmThreads) {
      const int rr = i % RPC, col = i / RPC;
      float acc = 0.f;
#pragma unroll
      for (int s = 0; s < KS; ++s) acc += recv[(s * RPC + rr) * L::RS + col];
      gemm_store<S>(p, j, dst_s, static_cast<int>(rank) * RPC + rr, col, acc);
    }
  }
  tc_fence_before();
  __syncthreads();
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc(tmem, L::TMEM_COLS);
  }
  // the launch before is waited for by one CTA: this grid cannot complete until that CTA
  // leaves, so kernels after it still find the earlier launch complete, while the short
  // jobs' CTAs leave their SMs at once (CTA 0 runs a value job, the longest)
  if (p.wait_at_exit && blockIdx.x == 0) griddep_wait();
}

// The values of many tokens on CTA pairs (tcgen05 cta_group::2), for appends whose keys go by
// rotproj.cu: D[256 ranks][NT tokens] = W_v rows x v tokens, K = H d.  Each CTA of a pair stages 128
// of the ranks and half of the tokens per k-block, for 256 tokens 32 KB where one CTA alone needs 48
// for half of the product, and has its 128 ranks of the accumulator for the epilogue above.  Bound by
// these copies (42 bytes a cycle and SM, 128 SMs 10 TB/s from L2), so 256 tokens where many tiles are
// to do, 128 where SMs would be idle.  (4096 tokens: the append 51.3 -> 45.5 us; plain appends keep
// keys and values in one launch of single CTAs.)
// KS: K in so many parts, a pair of CTAs each, in one cluster.  Each CTA finishes NT / KS of the tokens:
// it gives every other pair's CTA of its ranks the columns that one finishes, a copy per warp to its
// shared memory, and adds the parts in order.
template <class S, int NT, int KS>
struct PairSmem {
  static constexpr int STG = NT == 256 ? 6 : 8;
  static constexpr int HALF = 128 * 128, STAGE = HALF + NT / 2 * 128;   // ranks, tokens
  static constexpr int SL = NT / KS, PART = 32 * SL * 4;      // tokens that a CTA finishes; a warp's part
  static constexpr int SEND_OFF = 4 * kEpiWarpBytes;          // (over idle stages) [KS][4 warps] parts
  static constexpr int RECV_OFF = SEND_OFF + KS * 4 * PART;
  static constexpr int BAR_OFF = STG * STAGE;                 // full[S] (even CTA), empty[S], acc, parts[4]
  static constexpr int MISC_OFF = BAR_OFF + (2 * STG + 1 + 4) * 8;
  static constexpr int DST_OFF = (MISC_OFF + 8 + 7) / 8 * 8;
  static constexpr int RED_OFF = DST_OFF + NT * 8;            // 4-bit append: [4 warps][16]
  static constexpr int TOTAL = RED_OFF + 4 * 16 * 4;
  static constexpr int ALLOC = TOTAL + 1024;
  static_assert(DST_OFF % 8 == 0 && 4 * kEpiWarpBytes <= STAGE && SL % 16 == 0, "alignment, staging");
  static_assert(KS == 1 || RECV_OFF + KS * 4 * PART <= STG * STAGE, "the parts fit the stages");
  // more than half an SM's: the CTAs of a pair sit on two SMs
  static_assert(2 * ALLOC > 228 * 1024 && ALLOC <= 227 * 1024, "shared memory budget");
};

template <class S, int NT, int KS>
__global__ void __launch_bounds__(kGemmThreads, 1)
    value_pair_kernel(const __grid_constant__ CUtensorMap w_map, const __grid_constant__ CUtensorMap v_map,
                      const GemmParams p) {
  using L = PairSmem<S, NT, KS>;
  constexpr int STG = L::STG, KB = S::H * S::D / 64 / KS, SL = L::SL;   // k-blocks of a pair
  static_assert(S::H * S::D / 64 % KS == 0, "K in equal parts");
  extern __shared__ uint8_t smem_raw[];
  uint8_t* sm = reinterpret_cast<uint8_t*>(
      (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~static_cast<uintptr_t>(1023));
  uint64_t* full = reinterpret_cast<uint64_t*>(sm + L::BAR_OFF);
  uint64_t* empty = full + STG;
  uint64_t* accb = empty + STG;
  uint64_t* part_full = accb + 1;           // [4] a warp's parts from the other pairs
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(sm + L::MISC_OFF);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(sm + L::MISC_OFF + 4);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int cta = static_cast<int>(cluster_ctarank());
  const int rank = cta & 1, pair = cta >> 1;      // half of the pair (0 issues the MMAs), part of K
  const uint32_t lead = static_cast<uint32_t>(cta & ~1);
  constexpr int NM = S::R / 256;
  const int job = blockIdx.x / (2 * KS), kb0 = pair * KB;
  GemmJob j{};
  j.kind = 0;
  j.m0 = (job % NM) * 256 + rank * 128;   // this CTA's ranks
  j.n0 = (job / NM) * NT;                 // the pair's tokens

  if (threadIdx.x == 0) {
    for (int s = 0; s < STG; ++s) {
      mbar_init(&full[s], 1);
      mbar_init(&empty[s], 1);
    }
    mbar_init(accb, 1);
    for (int w = 0; w < 4; ++w) mbar_init(&part_full[w], 1);
    *abort_flag = 0;
    fence_mbar_init();
  }
  if (warp == 1) {
    tmem_alloc_pair(tmem_slot, NT);
    tmem_relinquish_pair();
  }
  tc_fence_before();
  cluster_sync_all();   // both CTAs' barriers exist before any copy reaches them
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;
  auto load = [&](int kb, bool a) {
    const int s = kb % STG;
    const uint32_t fb = map_to_rank(smem_u32(&full[s]), lead);
    if (a) {
      if (rank == 0) mbar_arrive_expect_tx(&full[s], 2 * L::STAGE);   // both CTAs' ranks and tokens
      tma_load_2d_pair(sm + s * L::STAGE, &w_map, (kb0 + kb) * 64, j.m0, fb);
    } else {
      tma_load_2d_pair(sm + s * L::STAGE + L::HALF, &v_map, (kb0 + kb) * 64, j.n0 + rank * (NT / 2), fb);
    }
  };
  // no kernel writes W_v: its first blocks do not wait for the launch ahead
  constexpr int PRE = KB < STG ? KB : STG;
  if (warp == 0 && lane == 0) {
    prefetch_tmap(&w_map);
    prefetch_tmap(&v_map);
    for (int kb = 0; kb < PRE; ++kb) load(kb, true);
  }
  if (!p.wait_at_exit) griddep_wait();
  griddep_launch();

  if (warp == 0 && lane == 0) {
    // ------------------------------------------------------------------------- copies
    int issued = PRE;
    for (int kb = 0; kb < PRE; ++kb) load(kb, false);
    for (int kb = PRE; kb < KB; ++kb) {
      if (!mbar_wait(&empty[kb % STG], ((kb / STG) - 1) & 1, abort_flag, p.dev_err)) break;
      load(kb, true);
      load(kb, false);
      issued = kb + 1;
    }
    // the last commits (arrivals on this CTA's barriers) land before it exits, and with them the
    // copies that they read
    for (int kb = issued - PRE; kb < issued; ++kb) mbar_wait_drain(&empty[kb % STG], (kb / STG) & 1);
  } else if (warp == 1 && lane == 0 && rank == 0) {
    // --------------------------------------------------------------------------- MMAs
    constexpr uint32_t idesc = make_idesc_f16(256, NT, false, false);
    int kb = 0;
    for (; kb < KB; ++kb) {
      const int s = kb % STG;
      if (!mbar_wait(&full[s], (kb / STG) & 1, abort_flag, p.dev_err)) break;
      tc_fence_after();
      const uint32_t a0 = smem_u32(sm + s * L::STAGE), b0 = a0 + L::HALF;
#pragma unroll
      for (int k = 0; k < 4; ++k)
        umma_f16_pair(tmem, make_sdesc(a0 + k * 32, 16, 1024, kSwizzle128B),
                      make_sdesc(b0 + k * 32, 16, 1024, kSwizzle128B), idesc,
                      (kb > 0 || k > 0) ? 1u : 0u);
      umma_commit_pair(&empty[s], static_cast<uint16_t>(0x3u << lead));
    }
    if (kb == KB) umma_commit_pair(accb, static_cast<uint16_t>(0x3u << lead));
    if (kb > 0) mbar_wait_drain(&empty[(kb - 1) % STG], ((kb - 1) / STG) & 1);
  }
  __syncwarp();
  int64_t* dst_s = reinterpret_cast<int64_t*>(sm + L::DST_OFF);
  for (int c = threadIdx.x; c < NT; c += kGemmThreads) dst_s[c] = append_dst<S>(p, j, c);
  __syncthreads();
  // ------------------------------------------------------------------------- epilogue
  const bool have_acc = __all_sync(0xffffffffu, mbar_wait(accb, 0, abort_flag, p.dev_err));
  tc_fence_after();
  const uint32_t trow = tmem + (static_cast<uint32_t>(warp * 32) << 16);
  uint8_t* stage = sm + warp * kEpiWarpBytes;   // (the pipeline's stages are idle)
  bool have = have_acc;
  if constexpr (KS > 1) {
    constexpr int CH = SL / 4;
    // pair to's part of this warp's rows: 16-byte chunk c of row `lane` at chunk c ^ (lane % CH)
    auto part = [&](int off, int to) { return sm + off + (to * 4 + warp) * L::PART; };
    auto chunk = [&](int c) { return (lane * CH + (c ^ (lane & (CH - 1)))) * 16; };
    if (lane == 0) mbar_arrive_expect_tx(&part_full[warp], (KS - 1) * L::PART);
    for (int to = 0; to < KS; ++to) {
      if (to == pair) continue;
#pragma unroll 1
      for (int c0 = 0; c0 < SL; c0 += 16) {
        float v[16];
        __syncwarp();
        tmem_ld16(trow + to * SL + c0, v);   // (no accumulator: what is there, and an error is set)
        tmem_wait_ld();
#pragma unroll
        for (int e = 0; e < 16; e += 4)
          *reinterpret_cast<float4*>(part(L::SEND_OFF, to) + chunk((c0 + e) / 4)) =
              make_float4(v[e], v[e + 1], v[e + 2], v[e + 3]);
      }
    }
    fence_proxy_async_smem();   // generic stores -> the copies' async-proxy reads
    cluster_sync_all();         // every CTA is done with its stages
    if (lane == 0)
      for (int to = 0; to < KS; ++to)
        if (to != pair) {
          const uint32_t other = static_cast<uint32_t>(2 * to + rank);
          bulk_s2peer(map_to_rank(smem_u32(part(L::RECV_OFF, pair)), other), part(L::SEND_OFF, to),
                      L::PART, map_to_rank(smem_u32(&part_full[warp]), other));
        }
    __syncwarp();
    have = __all_sync(0xffffffffu, mbar_wait(&part_full[warp], 0, abort_flag, p.dev_err)) && have;
  }
  auto blocks = [&](auto store) {
#pragma unroll 1
    for (int c0 = pair * SL; c0 < pair * SL + SL; c0 += 16) {
      float v[16];
      if (have) {
        tmem_ld16(trow + c0, v);
        tmem_wait_ld();
        if constexpr (KS > 1) {
          constexpr int CH = SL / 4;
          float sum[16];
#pragma unroll
          for (int from = 0; from < KS; ++from) {   // in order, whichever pair adds them
            const uint8_t* src = sm + L::RECV_OFF + (from * 4 + warp) * L::PART;
#pragma unroll
            for (int e = 0; e < 16; e += 4) {
              float4 x = make_float4(v[e], v[e + 1], v[e + 2], v[e + 3]);
              if (from != pair)
                x = *reinterpret_cast<const float4*>(
                    src + (lane * CH + (((c0 - pair * SL + e) / 4) ^ (lane & (CH - 1)))) * 16);
              sum[e] = from ? sum[e] + x.x : x.x;
              sum[e + 1] = from ? sum[e + 1] + x.y : x.y;
              sum[e + 2] = from ? sum[e + 2] + x.z : x.z;
              sum[e + 3] = from ? sum[e + 3] + x.w : x.w;
            }
          }
#pragma unroll
          for (int e = 0; e < 16; ++e) v[e] = sum[e];
        }
      } else {
#pragma unroll
        for (int e = 0; e < 16; ++e) v[e] = 0.f;
      }
      store(c0, v);
    }
  };
  if (p.fmt == RCP_PAGES_INT4)
    blocks([&](int c0, const float(&v)[16]) {
      int4_store_columns<S, 16>(p, j, dst_s, reinterpret_cast<float*>(sm + L::RED_OFF), c0, v);
    });
  else if (!have) {}
  else if (p.fmt == RCP_PAGES_FP8_E4M3)
    blocks([&](int c0, const float(&v)[16]) { gemm_store_block<S, 1, 1>(p, j, dst_s, stage, warp, lane, c0, v); });
  else
    blocks([&](int c0, const float(&v)[16]) { gemm_store_block<S, 2, 1>(p, j, dst_s, stage, warp, lane, c0, v); });
  tc_fence_before();
  cluster_sync_all();   // neither CTA leaves (or frees its columns) while the other is busy
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc_pair(tmem, NT);
  }
  if (p.wait_at_exit && blockIdx.x == 0) griddep_wait();
}

// --------------------------------------------------------------------------- launchers
template <class K>
static cudaError_t launch_cluster(K kernel, int grid, int cluster, int smem, cudaStream_t stream,
                                  bool pdl, const CUtensorMap& a, const CUtensorMap& a2,
                                  const CUtensorMap& b, const CUtensorMap& b2,
                                  const CUtensorMap& b3, const GemmParams& p) {
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3(grid);
  cfg.blockDim = dim3(kGemmThreads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = stream;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = cluster;
  attr[0].val.clusterDim.y = 1;
  attr[0].val.clusterDim.z = 1;
  attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[1].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = pdl ? 2 : 1;
  return cudaLaunchKernelEx(&cfg, kernel, a, a2, b, b2, b3, p);
}

// Append: small token counts split K over an 8-CTA cluster (64-token tiles); large ones
// use 256-token tiles without a split.
template <class S>
struct AppendCfg {
  static constexpr int KS_SMALL = (S::H * S::D / 64) < 8 ? (S::H * S::D / 64) : 8;
  // of rotated keys, where there are several tiles of 64 tokens: every job then finds its SMs at once
  // (128 tokens 15.8 -> 10.6 us, 192 16.6 -> 11.0).  Keys that come as they are keep the parts of a plain
  // append, whatever becomes of the queries beside them: a step stores what its append alone would
  static constexpr int KS_TILES = KS_SMALL < 4 ? KS_SMALL : 4;
  // pipeline stages by token tile: every k-block of a split-K value job (or of a key /
  // query job) in flight at once where shared memory allows
  static constexpr int STG16 = 8, STG64 = 6, STG256 = 4;
};

template <class S>
cudaError_t prepare_gemm() {
  cudaError_t e;
  auto set = [&](auto kernel, int smem) {
    cudaError_t r = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
    if (r == cudaSuccess)
      r = cudaFuncSetAttribute(kernel, cudaFuncAttributeNonPortableClusterSizeAllowed, 0);
    return r;
  };
  using AC = AppendCfg<S>;
  constexpr int KSS = AC::KS_SMALL;
  if ((e = set(gemm_kernel<S, kModeAppend, 16, KSS, AC::STG16>,
               GemmSmem<16, KSS, 1, AC::STG16>::ALLOC)) != cudaSuccess)
    return e;
  if ((e = set(gemm_kernel<S, kModeAppend, 64, KSS, AC::STG64>,
               GemmSmem<64, KSS, 1, AC::STG64>::ALLOC)) != cudaSuccess)
    return e;
  if ((e = set(gemm_kernel<S, kModeAppend, 256, 1, AC::STG256>,
               GemmSmem<256, 1, 1, AC::STG256>::ALLOC)) != cudaSuccess)
    return e;
  if ((e = set(gemm_kernel<S, kModeAppend, 16, KSS, AC::STG16, true>,
               GemmSmem<16, KSS, 1, AC::STG16>::ALLOC)) != cudaSuccess)
    return e;
  if ((e = set(gemm_kernel<S, kModeAppend, 64, KSS, AC::STG64, true>,
               GemmSmem<64, KSS, 1, AC::STG64>::ALLOC)) != cudaSuccess)
    return e;
  if ((e = set(gemm_kernel<S, kModeAppend, 64, AC::KS_TILES, AC::STG64, true>,
               GemmSmem<64, AC::KS_TILES, 1, AC::STG64>::ALLOC)) != cudaSuccess)
    return e;
  if constexpr (S::R % 256 == 0) {
    if ((e = set(value_pair_kernel<S, 256, 1>, PairSmem<S, 256, 1>::ALLOC)) != cudaSuccess) return e;
    if ((e = set(value_pair_kernel<S, 128, 1>, PairSmem<S, 128, 1>::ALLOC)) != cudaSuccess) return e;
    if ((e = set(value_pair_kernel<S, 128, 2>, PairSmem<S, 128, 2>::ALLOC)) != cudaSuccess) return e;
    if ((e = set(value_pair_kernel<S, 128, 4>, PairSmem<S, 128, 4>::ALLOC)) != cudaSuccess) return e;
  }
  if ((e = set(gemm_kernel<S, kModeQproj, 64, 1, 2>, GemmSmem<64, 1, 1, 2>::ALLOC)) != cudaSuccess)
    return e;
  if ((e = set(gemm_kernel<S, kModeQproj, 256, 1, 2>, GemmSmem<256, 1, 1, 2>::ALLOC)) != cudaSuccess)
    return e;
  return cudaSuccess;
}

// The append's projections and, when ap.nq > 0, the rank-space queries (a decode's, or a
// chunked prefill step's when ap.qhi is set), in one launch (either part may be empty), or, with more
// than 192 rows of which some are rotated, two.  q_rows: tensor map over the queries [nq][H*d]; the
// boxes of all maps as launch.h has them.
template <class S>
cudaError_t launch_append_gemm(const CUtensorMap& w_v, const CUtensorMap& u_k,
                               const CUtensorMap& v_rows, const CUtensorMap& k_rows,
                               const CUtensorMap& q_rows, const AppendParams& ap,
                               cudaStream_t stream) {
  if (ap.T == 0 && ap.nq == 0) return cudaSuccess;
  GemmParams p{};
  p.slots = ap.slots;
  p.k_pages = ap.k_pages;
  p.v_pages = ap.v_pages;
  p.T = ap.T;
  p.fmt = ap.page_format;
  p.num_blocks = ap.num_blocks;
  p.dev_err = ap.dev_err;
  p.qt = ap.qt;
  p.qhi = ap.qhi;
  p.qlo = ap.qlo;
  p.nq = ap.nq;
  p.qscale = ap.qscale;
  p.wait_at_exit = ap.wait_at_exit;
  using AC = AppendCfg<S>;
  constexpr int NM = (S::R + 127) / 128;
  constexpr int KS = AC::KS_SMALL;
  constexpr int NKG = (S::H / 2 + KS - 1) / KS;
  const int rows = ap.T > ap.nq ? ap.T : ap.nq;
  const bool rot = ap.rot_table != nullptr;
  p.rot_table = ap.rot_table;
  p.k_pos = ap.k_pos;
  p.q_pos = ap.q_pos;
  p.num_pos = ap.num_pos;
  p.rot_dim = ap.rot_dim;
  p.interleaved = ap.interleaved;
  auto go = [&](auto kernel, int clusters, int cluster, int smem) {
    return launch_cluster(kernel, clusters * cluster, cluster, smem, stream, true, w_v, u_k, v_rows,
                          k_rows, q_rows, p);
  };
  if (rows <= 16) {   // a decode step of up to 16 requests: 16-row tiles
    const int clusters = (ap.T + 15) / 16 * (NM + NKG) + (ap.nq + 15) / 16 * NKG;
    constexpr int smem = GemmSmem<16, KS, 1, AC::STG16>::ALLOC;
    return rot ? go(gemm_kernel<S, kModeAppend, 16, KS, AC::STG16, true>, clusters, KS, smem)
               : go(gemm_kernel<S, kModeAppend, 16, KS, AC::STG16>, clusters, KS, smem);
  }
  if (ap.value_tile == 0 && rows <= 256) {
    if (ap.k_pos != nullptr && ap.T > 64) {
      constexpr int KT = AC::KS_TILES, NKT = (S::H / 2 + KT - 1) / KT;
      return go(gemm_kernel<S, kModeAppend, 64, KT, AC::STG64, true>,
                (ap.T + 63) / 64 * (NM + NKT) + (ap.nq + 63) / 64 * NKT, KT,
                GemmSmem<64, KT, 1, AC::STG64>::ALLOC);
    }
    const int clusters = (ap.T + 63) / 64 * (NM + NKG) + (ap.nq + 63) / 64 * NKG;
    constexpr int smem = GemmSmem<64, KS, 1, AC::STG64>::ALLOC;
    return rot ? go(gemm_kernel<S, kModeAppend, 64, KS, AC::STG64, true>, clusters, KS, smem)
               : go(gemm_kernel<S, kModeAppend, 64, KS, AC::STG64>, clusters, KS, smem);
  }
  // many tokens or queries: 256-row tiles, no split.  Rotated: the values alone, keys and queries
  // behind them (rotproj.cu)
  constexpr int smem = GemmSmem<256, 1, 1, AC::STG256>::ALLOC;
  const int tiles = (ap.T + 255) / 256, qtiles = (ap.nq + 255) / 256;
  if (rot) {
    p.nq = 0;
    if (ap.T > 0) {
      cudaError_t e;
      if constexpr (S::R % 256 == 0) {
        auto pairs = [&](auto kernel, int smem) {
          cudaLaunchConfig_t cfg{};
          cfg.gridDim = dim3((ap.T + ap.value_tile - 1) / ap.value_tile * (S::R / 256) * 2 * ap.value_splits);
          cfg.blockDim = dim3(kGemmThreads);
          cfg.dynamicSmemBytes = smem;
          cfg.stream = stream;
          cudaLaunchAttribute attr[2];
          attr[0].id = cudaLaunchAttributeClusterDimension;
          attr[0].val.clusterDim.x = 2 * ap.value_splits;
          attr[0].val.clusterDim.y = 1;
          attr[0].val.clusterDim.z = 1;
          attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
          attr[1].val.programmaticStreamSerializationAllowed = 1;
          cfg.attrs = attr;
          cfg.numAttrs = 2;
          return cudaLaunchKernelEx(&cfg, kernel, w_v, v_rows, p);
        };
        e = ap.value_splits == 4   ? pairs(value_pair_kernel<S, 128, 4>, PairSmem<S, 128, 4>::ALLOC)
            : ap.value_splits == 2 ? pairs(value_pair_kernel<S, 128, 2>, PairSmem<S, 128, 2>::ALLOC)
            : ap.value_tile == 128 ? pairs(value_pair_kernel<S, 128, 1>, PairSmem<S, 128, 1>::ALLOC)
                                   : pairs(value_pair_kernel<S, 256, 1>, PairSmem<S, 256, 1>::ALLOC);
      } else {
        e = go(gemm_kernel<S, kModeAppend, 256, 1, AC::STG256>, tiles * NM, 1, smem);
      }
      if (e != cudaSuccess) return e;
    }
    return launch_rotated_proj<S>(u_k, k_rows, q_rows, ap, ap.T > 0, stream);
  }
  return go(gemm_kernel<S, kModeAppend, 256, 1, AC::STG256>,
            tiles * (NM + S::H / 2) + qtiles * (S::H / 2), 1, smem);
}

template <class S>
cudaError_t launch_qproj_gemm(const CUtensorMap& u_k, const CUtensorMap& q_rows, void* qhi,
                              void* qlo, int nq, float qscale, uint32_t* dev_err,
                              cudaStream_t stream, bool pdl) {
  GemmParams p{};
  p.nq = nq;
  p.qhi = qhi;
  p.qlo = qlo;
  p.qscale = qscale;
  p.dev_err = dev_err;
  if (nq <= 256) {
    const int tiles = (nq + 63) / 64;
    return launch_cluster(gemm_kernel<S, kModeQproj, 64, 1, 2>, tiles * (S::H / 2), 1,
                          GemmSmem<64, 1, 1, 2>::ALLOC, stream, pdl, u_k, u_k, q_rows, q_rows,
                          q_rows, p);
  }
  const int tiles = (nq + 255) / 256;
  return launch_cluster(gemm_kernel<S, kModeQproj, 256, 1, 2>, tiles * (S::H / 2), 1,
                        GemmSmem<256, 1, 1, 2>::ALLOC, stream, pdl, u_k, u_k, q_rows, q_rows,
                        q_rows, p);
}

template cudaError_t prepare_gemm<ShapeMain>();
template cudaError_t prepare_gemm<ShapeTiny>();
template cudaError_t launch_append_gemm<ShapeMain>(const CUtensorMap&, const CUtensorMap&,
                                                   const CUtensorMap&, const CUtensorMap&,
                                                   const CUtensorMap&, const AppendParams&,
                                                   cudaStream_t);
template cudaError_t launch_append_gemm<ShapeTiny>(const CUtensorMap&, const CUtensorMap&,
                                                   const CUtensorMap&, const CUtensorMap&,
                                                   const CUtensorMap&, const AppendParams&,
                                                   cudaStream_t);
template cudaError_t launch_qproj_gemm<ShapeMain>(const CUtensorMap&, const CUtensorMap&, void*,
                                                  void*, int, float, uint32_t*, cudaStream_t,
                                                  bool);
template cudaError_t launch_qproj_gemm<ShapeTiny>(const CUtensorMap&, const CUtensorMap&, void*,
                                                  void*, int, float, uint32_t*, cudaStream_t,
                                                  bool);

}  // namespace rcp
