// Chunked-prefill attention over low-rank paged coefficients on tensor cores.
//
// The "Per-prefill-chunk attention" step of the Proxima page: every row i of a request's
// chunk (absolute position P + i) attends keys 0 .. P + i of the paged cache, after the
// chunk itself has been appended.  The scores are rank-space products and the values a
// joint coefficient contraction, so one CTA owns (request, head h, 128 query rows, one
// slice of up to 256 of the R joint ranks) and walks the causal key range in tiles of
// 128 tokens (8 pages):
//
//   S   = Q~_h C_k,h^T          tcgen05, M=128 rows x N=128 keys x K=64 (q~ as fp16 hi+lo)
//   P   = exp2(S - m)           one thread per query row (TMEM lane), lazy rescaling
//   Z  += P C_v[:, slice]       tcgen05, M=128 x N=256 x K=128, accumulator in TMEM
//
// S is double-buffered in TMEM so the score MMA of tile j+1 overlaps the softmax of tile
// j, and the softmax of tile j overlaps the value MMA of tile j-1.  At the end each row
// is normalised, split into an fp16 (hi, lo) pair and multiplied by the slice's rows of
// W_v[:, h*d:(h+1)*d] (tcgen05 again); the slices of one (request, head, tile) form a
// thread-block cluster and sum their partial outputs through distributed shared memory.
//
// The reconstructing variant (RECON) attends V^ = C_v W_v rows of head h, rebuilt once per
// key by the reconstruction GEMM: O += P V^_h (M=128 x N=d x K=128) in TMEM, no rank slices,
// and the softmax warps write O / l straight to the output; its key/value ring has three
// stages, and P stays in tensor memory (two buffers, stored by the softmax threads with
// tcgen05.st and read as the value MMA's A operand).
//
// Warps: 0 copies queries and key tiles, 6 copies value tiles and the W_v slice (two
// independent streams: a key stage is freed by its score MMA, a value stage by its value
// MMA), 1 issues the MMAs (and owns TMEM), 2-5 run the softmax and the epilogue (warp w
// serves TMEM lanes 32*(w%4) .. +31).
//
// Roundings: the scores, the running maximum and sum and the accumulators are fp32; the weights
// enter the value MMA in fp16 (kind::f16 takes both operands in 16 bits), V^ is stored in fp16
// by the reconstruction.  Each moves the output by 2.0e-4 of its norm, its own rounding to fp16
// by 2.1e-4, together 3.5e-4; a second fp16 term of either would double the value product or
// the V^ traffic.
//
// MOD (score modifications, scoremod.cuh): eight softmax warps, 2-9, two threads per row with 64
// keys of a tile each, because one warp per scheduler cannot hide the arithmetic added to every
// score (16 x (4096 + 256), cap + bias: 1071 -> 914 us); the value copies are warp 10's.  The
// key tiles are those that some row of the CTA sees, the nearest first.  Measured per tile
// (cycles): 2500 with masks alone, 3600 with a cap (FMA pipe), plain 2210; whole calls 0.87 ms
// with cap and bias and 0.76 ms with masks, plain 0.70 ms.
#include <cuda.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include <cstdint>
#include <type_traits>

#include "launch.h"
#include "ptx.cuh"
#include "rcp.h"
#include "scoremod.cuh"
#include "shape.h"

namespace rcp {

// Warps: 0 key copies, 1 MMAs, then the softmax warps and one for the value copies.
//   plain  2-5 softmax (one thread per query row), 6 value copies
//   MOD    2-9 softmax (two threads per row, each with half of a tile's keys), 10
template <bool MOD>
struct PfWarps {
  static constexpr int NSW = MOD ? 8 : 4;
  static constexpr int THREADS = 32 * (3 + NSW);
};
constexpr float kPfRescale = 8.f;   // log2 units: weights stay below 2^8 between rescales

// RECON: the values are the reconstructed V^ rows of head h (N = d) instead of a slice
// of the joint coefficients (N = RQ), and the epilogue writes O directly.
template <class S, bool RECON, bool MOD = false, bool PERS = false>
struct PfSmem {
  using C = PrefillCfg<S>;
  static constexpr int VN = RECON ? S::D : C::RQ;       // value MMA N
  static constexpr int NQ = RECON ? 1 : C::NQ;          // CTAs per (tile, head)
  static constexpr int NG = VN / 64;                    // 64-wide groups of the value tile
  static constexpr int Q_BYTES = 128 * 128;             // one [128][64] fp16 operand
  static constexpr int K_BYTES = C::KT * 128;           // key coefficients of one tile
  static constexpr int V_BYTES = C::KT * VN * 2;        // value tile
  static constexpr int STAGE = K_BYTES + V_BYTES;
  static constexpr int NS = RECON ? 3 : 2;              // key/value pipeline stages
  // RECON keeps P in tensor memory (two buffers at columns P_TM and P_TM + KT/2, the A
  // operand of the value MMA); the rank-space variant stages it in shared memory
  static constexpr int P_BYTES = RECON ? 0 : 128 * C::KT * 2;
  static constexpr int P_TM = 256 + VN;
  static_assert(!PERS || (RECON && MOD), "variants");
  static constexpr int QB = PERS ? 2 : 1;               // query buffers (this item, the next)
  static constexpr int ST_OFF = QB * 2 * Q_BYTES;       // q~ hi at 0, q~ lo at Q_BYTES
  static constexpr int P_OFF = ST_OFF + NS * STAGE;
  static constexpr int ZH_OFF = ST_OFF;                 // epilogue reuses the stage memory
  static constexpr int ZL_OFF = ZH_OFF + 128 * C::RQ * 2;
  static constexpr int W_OFF = ZL_OFF + 128 * C::RQ * 2;
  static constexpr int W_BYTES = C::RQ * S::D * 2;
  static constexpr int END = (RECON || P_OFF + P_BYTES > W_OFF + W_BYTES) ? P_OFF + P_BYTES
                                                                             : W_OFF + W_BYTES;
  static constexpr int NBAR = 11 + 4 * NS + (PERS ? 7 : 0);
  static constexpr int BAR_OFF = END;                   // NBAR mbarriers
  static constexpr int MISC_OFF = BAR_OFF + NBAR * 8;   // tmem slot, abort flag
  // MOD: least and largest first token of the tile's rows (per warp), the rejected pages of
  // each key stage and of each score buffer, the softmax warps' column masks [2][4][4] and the
  // row halves' maxima [HB][2][128] (the rank-space variant has room for one buffer).
  // PERS: the row halves' sums [2][128] and two work items
  static constexpr int MOD_OFF = MISC_OFF + 16;
  static constexpr int HB = RECON ? 2 : 1;
  static constexpr int ITEM = 12;                       // ints of a work item
  static constexpr int MOD_BYTES =
      (MOD ? (8 + 8 + 2 + 2 * 16 + HB * 2 * 128) * 4 : 0) + (PERS ? (2 * 128 + 2 * ITEM) * 4 : 0);
  static constexpr int TOTAL = MOD_OFF + MOD_BYTES;
  static constexpr int ALLOC = TOTAL + 1024;
  static constexpr int RPC = 128 / NQ;                  // output rows each slice CTA sums
  static constexpr int TMEM_COLS = pow2_at_least(256 + VN, 32);
  static_assert(ALLOC <= 227 * 1024, "shared memory budget");
  static_assert(NQ == 1 || NQ * RPC * S::D * 4 <= 2 * 128 * C::RQ * 2, "receive buffer");
  static_assert(256 + VN <= 512 && S::D <= 128, "tensor memory budget");
  static_assert(!RECON || P_TM + C::KT <= TMEM_COLS, "P buffers in tensor memory");
};

// MOD: score modifications (rcp_score_mod).  A row sees keys t < pfx and lo <= t <= pos with
// its own lo, so the CTA walks the key tiles of the prefix and those from the least lo of
// its rows on; each row masks its scores to what it sees, and a key that no row of the tile
// sees has its value row zeroed.
//
// PERS (MOD with RECON, launch_prefill's rule): one CTA per SM takes (query tile, head) items
// until none is left, from a counter that the plan resets.  The key warp works out the next
// item and loads its queries and first keys, and its first scores are computed, while the
// softmax warps finish this one.  A CTA per item spends 10,000 cycles on starting and ending,
// as much as four key tiles: packed documents of about 700 tokens, 2 x 4096, 274 -> 238 us.
template <class S, bool RECON, bool MOD, bool PERS>
__global__ void __launch_bounds__(PfWarps<MOD>::THREADS, 1)
    prefill_kernel(const __grid_constant__ CUtensorMap qhi_map,
                   const __grid_constant__ CUtensorMap qlo_map,
                   const __grid_constant__ CUtensorMap kp_map,
                   const __grid_constant__ CUtensorMap vp_map,
                   const __grid_constant__ CUtensorMap w_map,
                   const __grid_constant__ AttnParams p) {
  using C = PrefillCfg<S>;
  using L = PfSmem<S, RECON, MOD, PERS>;
  constexpr int KT = C::KT, RQ = C::RQ, NQ = L::NQ, NG = L::NG, VN = L::VN, D = S::D, H = S::H;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* sm = reinterpret_cast<uint8_t*>(
      (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~static_cast<uintptr_t>(1023));
  uint64_t* bars = reinterpret_cast<uint64_t*>(sm + L::BAR_OFF);
  constexpr int NS = L::NS;
  uint64_t* q_full = bars + 0;
  uint64_t* k_full = bars + 1;              // [NS] key half of a stage landed
  uint64_t* v_full = k_full + NS;           // [NS] value half of a stage landed
  uint64_t* k_empty = v_full + NS;          // [NS] score MMA of the stage's tile done
  uint64_t* v_empty = k_empty + NS;         // [NS] value MMA of the stage's tile done
  uint64_t* s_full = v_empty + NS;          // [2] scores of a tile in TMEM
  uint64_t* p_full = s_full + 2;            // [2] softmax weights written (4 warps)
  uint64_t* pv_done = p_full + 2;           // [2] value MMA of a P buffer done
  uint64_t* acc_done = pv_done + 2;
  uint64_t* zq_full = acc_done + 1;
  uint64_t* w_full = zq_full + 1;
  uint64_t* o_done = w_full + 1;
  uint64_t* q_empty = o_done + 1;           // PERS [2] a query buffer is no longer used
  uint64_t* item_full = q_empty + 2;        // PERS [2] a work item is written
  uint64_t* item_empty = item_full + 2;     // PERS [2] ... and read by every warp that does
  uint64_t* q_full2 = item_empty + 2;       // PERS: of the second query buffer
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(sm + L::MISC_OFF);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(sm + L::MISC_OFF + 4);
  // MOD: by a shuffle, which tells the compiler that a warp's role is uniform (16 x (4096 + 256),
  // cap + bias: 881 -> 865 us)
  const int warp = MOD ? __shfl_sync(0xffffffffu, threadIdx.x >> 5, 0) : threadIdx.x >> 5;
  const int lane = threadIdx.x & 31;

  griddep_wait();            // plan and rank-space queries are ready
  const int slice = blockIdx.x % NQ;                    // cluster rank when NQ > 1
  if (!PERS && blockIdx.x / (H * NQ) >= *p.tcount) return;   // uniform over the cluster
  // the (query tile, head) of this CTA; PERS: of the item that this warp is at
  int h = 0, b = 0, n = 0, P0 = 0, nkt = 0, nblk = 0, i0 = 0, row0 = 0, Lb = 0;
  auto locate = [&](int slot) {
    b = p.tile_b[slot];
    i0 = p.tile_qt[slot] * 128;                         // first chunk row of this tile
    const int c0 = p.cu_chunk[b];
    n = p.cu_chunk[b + 1] - c0;
    Lb = p.seq_lens[b];
    P0 = Lb - n;
    nkt = (P0 + min(n, i0 + 128) - 1 + KT) / KT;        // key tiles (causal limit)
    nblk = (Lb + kBlockSize - 1) / kBlockSize;
    row0 = c0 + i0;
  };
  if constexpr (!PERS) {
    h = (blockIdx.x / NQ) % H;
    locate(blockIdx.x / (H * NQ));
  }
  int* wlo = reinterpret_cast<int*>(sm + L::MOD_OFF);   // MOD [8]: least, largest lo per warp
  int* kbad = wlo + 8;                                  // MOD [8]: rejected pages of a tile
  int* sbad = kbad + 8;                                 // MOD [2]: the same per score buffer
  uint32_t* colm = reinterpret_cast<uint32_t*>(sbad + 2);   // MOD [2][4][4]
  float* half_max = reinterpret_cast<float*>(colm + 32);    // MOD [HB][2][128]
  float* half_sum = half_max + (PERS ? L::HB * 256 : 0);    // MOD [2][128]
  int* items = reinterpret_cast<int*>(half_sum + 256);      // PERS [2][ITEM]
  using W = PfWarps<MOD>;
  constexpr int NSW = W::NSW;                               // softmax warps 2 .. NSW + 1
  constexpr int HALVES = NSW / 4;                           // threads per query row

  if (threadIdx.x == 0) {
    mbar_init(q_full, 1);
    for (int s = 0; s < NS; ++s) {
      mbar_init(&k_full[s], 1);
      mbar_init(&v_full[s], 1);
      mbar_init(&k_empty[s], 1);
      mbar_init(&v_empty[s], 1);
    }
    mbar_init(&s_full[0], MOD ? 2 : 1);   // the commit (MOD: and the MMA thread, after sbad)
    mbar_init(&s_full[1], MOD ? 2 : 1);
    for (int i = 0; i < 2; ++i) {
      mbar_init(&p_full[i], NSW);
      mbar_init(&pv_done[i], 1);
    }
    mbar_init(acc_done, 1);
    mbar_init(zq_full, NSW);
    mbar_init(w_full, 1);
    mbar_init(o_done, 1);
    if constexpr (PERS) {
      for (int i = 0; i < 2; ++i) {
        mbar_init(&q_empty[i], 1 + NSW);      // its last score MMA, the softmax warps
        mbar_init(&item_full[i], 1);
        mbar_init(&item_empty[i], 2 + NSW);   // the MMA, value-copy and softmax warps
      }
      mbar_init(q_full2, 1);
    }
    *abort_flag = 0;
    fence_mbar_init();
  }
  if (warp == 1) {
    tmem_alloc(tmem_slot, L::TMEM_COLS);
    tmem_relinquish();
  }
  // MOD: rows of this tile by thread, their first tokens; rows past the chunk do not count
  if constexpr (MOD && !PERS) {
    if (warp < 4) {
      const int ci = i0 + static_cast<int>(threadIdx.x);
      const int32_t f = ci < n ? view_begin(p, row0 - i0 + ci, P0 + ci) : 0;
      const int32_t least = __reduce_min_sync(0xffffffffu, ci < n && f <= P0 + ci ? f : INT32_MAX);
      const int32_t most = __reduce_max_sync(0xffffffffu, ci < n ? f : 0);
      if (lane == 0) {
        wlo[warp] = least;
        wlo[4 + warp] = most;
      }
    }
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  // only now: the next launch's CTAs, which hold tensor memory while they wait for this one,
  // must not take this CTA's place in it
  griddep_launch();
  const uint32_t tmem = *tmem_slot;
  int32_t pfx = 0, lo_min = 0, lo_max = 0, npt = 0, lt = 0;   // MOD: tiles [0, npt), then lt ..
  auto tiles_seen = [&](int least, int most) {
    pfx = view_prefix(p, b, Lb);
    lo_min = least;
    lo_max = most;
    npt = (pfx + KT - 1) / KT;
    lt = lo_min < INT32_MAX ? lo_min / KT : nkt;
    lt = max(lt, npt);
    nkt = npt + max(0, nkt - lt);
  };
  if constexpr (MOD && !PERS)
    tiles_seen(min(min(wlo[0], wlo[1]), min(wlo[2], wlo[3])),
               max(max(wlo[4], wlo[5]), max(wlo[6], wlo[7])));
  // PERS: this warp's next item, number it; false: none is left (or a wait failed).  softmax: the
  // softmax warps take it or leave it together, because they meet at barriers in its tiles,
  // which a warp whose wait has failed would miss; and a warp's lanes read it together, which
  // the reductions tell the compiler (loops over the item's tiles stay in uniform registers)
  auto take_item = [&](int it, auto softmax) {
    bool ok = mbar_wait(&item_full[it & 1], (it >> 1) & 1, abort_flag, p.dev_err);
    if constexpr (decltype(softmax)::value) ok = named_bar_and(1, 32 * NSW, ok);
    const int* m = items + (it & 1) * L::ITEM;
    auto get = [&](int x) {
      if constexpr (decltype(softmax)::value) return __reduce_max_sync(0xffffffffu, x);
      else return x;
    };
    nkt = get(ok ? m[0] : -1);
    b = get(m[1]);
    h = get(m[2]);
    row0 = get(m[3]);
    i0 = get(m[4]);
    n = get(m[5]);
    P0 = get(m[6]);
    nblk = get(m[7]);
    pfx = get(m[8]);
    lo_max = get(m[9]);
    lt = get(m[10]);
    npt = (pfx + KT - 1) / KT;
    return nkt >= 0;
  };
  // key tile number j of this CTA.  MOD: the nearest first, so that under a bias the running
  // maximum settles with the first tile (it would grow, and the accumulator be rescaled, with
  // every tile that comes nearer)
  auto tile_of = [&](int j) {
    if (!MOD) return j;
    const int i = nkt - 1 - j;
    return i >= npt ? lt + (i - npt) : i;
  };
  // whether page x of the request is read (MOD: some row of the tile may see it)
  auto page_read = [&](int x) {
    return x < nblk && (!MOD || x * kBlockSize < pfx || (x + 1) * kBlockSize > lo_min);
  };
  if constexpr (NQ > 1) cluster_sync_all();   // peers are running before any remote store

  // MOD: a tile that every row of the CTA sees whole needs no mask
  auto sees_whole = [&](int t0, uint32_t bad) {
    return bad == 0 && (t0 + KT <= pfx || (lo_max <= t0 && t0 + KT - 1 <= P0 + i0));
  };
  // MOD: zeroes the value rows of tile g's keys whose bit is set, by nt threads (this one: tid)
  auto zero_values = [&](int g, const uint32_t (&keys)[4], int tid, int nt) {
    uint8_t* vst = sm + L::ST_OFF + (g % NS) * L::STAGE + L::K_BYTES;
    for (int idx = tid; idx < KT * NG * 8; idx += nt) {
      const int tok = idx / (NG * 8);
      const uint32_t w = tok < 64 ? (tok < 32 ? keys[0] : keys[1]) : (tok < 96 ? keys[2] : keys[3]);
      if (!((w >> (tok & 31)) & 1u)) continue;
      const int rem = idx % (NG * 8);
      const int box = rem >> 3, ch = rem & 7;
      *reinterpret_cast<uint4*>(vst + (box * (KT / kBlockSize) + tok / kBlockSize) * 2048 +
                                (tok % kBlockSize) * 128 + ch * 16) = make_uint4(0, 0, 0, 0);
    }
  };
  // A warp whose copies or MMAs may still be under way when it has nothing left to do (a wait
  // failed somewhere) stays until they are done: this CTA's memory is another's once it has
  // left.  n tiles' copies in all, the last NS of which may be on their way.
  auto drain_copies = [&](uint64_t* full, int n) {
    for (int i = max(0, n - NS); i < n; ++i) mbar_wait_drain(&full[i % NS], (i / NS) & 1);
  };
  if (warp == 0) {
    // ------------------------------------------------------------------ key copies
    // The whole warp: lane jb < 8 resolves page jb of each tile one tile ahead and issues
    // that page's copy (the eight small copies of a tile set the kernel's pace when one
    // thread issues them in turn); lane 0 waits for the stage and arms its byte count.
    constexpr int BPT = KT / kBlockSize;                  // pages per key tile
    if (lane == 0) prefetch_tmap(&kp_map);
    auto load_queries = [&](int qb, uint64_t* full) {
      mbar_arrive_expect_tx(full, 2 * L::Q_BYTES);
      tma_load_2d(sm + qb * 2 * L::Q_BYTES, &qhi_map, h * 64, row0, full);
      tma_load_2d(sm + qb * 2 * L::Q_BYTES + L::Q_BYTES, &qlo_map, h * 64, row0, full);
    };
    if (!PERS && lane == 0) load_queries(0, q_full);
    bool ok = true;
    [[maybe_unused]] int nq = 0;                          // PERS: items with key tiles
    int issued = 0;                                       // tiles whose copies are under way or done
    for (int it = 0, g0 = 0; ok; ++it) {                  // g0: tiles of the items before
      if constexpr (PERS) {
        int w = blockIdx.x;
        if (it > 0) {
          if (lane == 0) w = gridDim.x + atomicAdd(p.tcount + 1, 1);
          w = __shfl_sync(0xffffffffu, w, 0);
        }
        const bool more = w / H < *p.tcount;
        if (more) {
          h = w % H;
          locate(w / H);
          int32_t least = INT32_MAX, most = 0;
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            const int r = 32 * k + lane;
            const int32_t f = i0 + r < n ? view_begin(p, row0 + r, P0 + i0 + r) : 0;
            if (i0 + r < n && f <= P0 + i0 + r) least = min(least, f);
            most = max(most, f);
          }
          tiles_seen(__reduce_min_sync(0xffffffffu, least), __reduce_max_sync(0xffffffffu, most));
        } else {
          nkt = -1;
        }
        if (it >= 2)
          ok = __all_sync(0xffffffffu, mbar_wait(&item_empty[it & 1], ((it - 2) >> 1) & 1,
                                                 abort_flag, p.dev_err));
        if (!ok) break;
        if (lane == 0) {
          int* m = items + (it & 1) * L::ITEM;
          const int v[L::ITEM] = {nkt, b, h, row0, i0, n, P0, nblk, pfx, lo_max, lt, nq};
#pragma unroll
          for (int k = 0; k < L::ITEM; ++k) m[k] = v[k];
          mbar_arrive(&item_full[it & 1]);
        }
        if (!more) break;
        if (nkt == 0) continue;
        if (nq >= 2)
          ok = __all_sync(0xffffffffu, mbar_wait(&q_empty[nq & 1], ((nq - 2) >> 1) & 1, abort_flag,
                                                 p.dev_err));
        if (!ok) break;
        if (lane == 0) load_queries(nq & 1, nq & 1 ? q_full2 : q_full);
        ++nq;
      }
      const int32_t* table = p.block_table + static_cast<int64_t>(b) * p.bt_stride;
      const int pg0 = tile_of(0) * BPT + lane;
      int32_t nxt = (lane < BPT && nkt > 0 && page_read(pg0)) ? table[pg0] : -1;
      for (int j = 0; ok && j < nkt; ++j) {
        const int g = g0 + j, s = g % NS;
        const bool mine = lane < BPT && page_read(tile_of(j) * BPT + lane);
        int32_t phys = mine ? nxt : -1;
        if (mine && (phys < 0 || phys >= p.num_blocks)) {
          atomicOr(p.dev_err, RCP_DEVERR_BAD_BLOCK);
          phys = -1;
        }
        const int nb = tile_of(j + 1) * BPT + lane;        // the next tile's page, in flight
        nxt = (lane < BPT && j + 1 < nkt && page_read(nb)) ? table[nb] : -1;
        // MOD: rejected pages, for the softmax to mask (keys run at most NS + 2 tiles ahead of it)
        const uint32_t rejected = MOD ? __ballot_sync(0xffffffffu, mine && phys < 0) : 0;
        const int nload = __popc(__ballot_sync(0xffffffffu, phys >= 0));
        if (lane == 0) {
          ok = g < NS || mbar_wait(&k_empty[s], ((g / NS) - 1) & 1, abort_flag, p.dev_err);
          if constexpr (MOD) kbad[g & 7] = static_cast<int>(rejected);
          if (ok) mbar_arrive_expect_tx(&k_full[s], nload * 2048);
        }
        ok = __shfl_sync(0xffffffffu, ok, 0);             // the byte count is armed first
        if (ok) issued = g + 1;
        if (ok && phys >= 0)
          tma_load_2d(sm + L::ST_OFF + s * L::STAGE + lane * 2048, &kp_map, 0,
                      (phys * H + h) * kBlockSize, &k_full[s]);
      }
      g0 += nkt;
      if constexpr (!PERS) break;
    }
    if (lane == 0) {
      drain_copies(k_full, issued);
      if constexpr (!PERS) mbar_wait_drain(q_full, 0);
      if (PERS && nq > 0) mbar_wait_drain(nq & 1 ? q_full : q_full2, ((nq - 1) >> 1) & 1);
      if (PERS && nq > 1) mbar_wait_drain(nq & 1 ? q_full2 : q_full, ((nq - 2) >> 1) & 1);
    }
  } else if (warp == 2 + NSW) {
    // ---------------------------------------------------------------- value copies
    if constexpr (RECON) {
      // V^ rows of the request are contiguous: one 64-column box of 128 keys per group
      if (lane == 0) {
        prefetch_tmap(&vp_map);
        bool ok = true;
        int issued = 0;
        for (int it = 0, g0 = 0; ok; ++it) {
          if constexpr (PERS) {
            if (!take_item(it, std::false_type{})) break;
            mbar_arrive(&item_empty[it & 1]);
          }
          const int64_t first = p.vcum[b] * kBlockSize;
          int tile0 = 0;                                // MOD: the tiles between npt and lt
          if constexpr (MOD) {                          // ... are not in V^
            const TileMap<S> map(p.vmap + 2 * b, nblk);
            tile0 = map.lt - map.np;
          }
          for (int j = 0; j < nkt; ++j) {
            const int g = g0 + j, s = g % NS;
            uint8_t* vst = sm + L::ST_OFF + s * L::STAGE + L::K_BYTES;
            ok = g < NS || mbar_wait(&v_empty[s], ((g / NS) - 1) & 1, abort_flag, p.dev_err);
            if (!ok) break;
            mbar_arrive_expect_tx(&v_full[s], NG * KT * 128);
            issued = g + 1;
            const int x = tile_of(j);
            const int64_t vrow = first + static_cast<int64_t>(MOD && x >= npt ? x - tile0 : x) * KT;
#pragma unroll
            for (int q = 0; q < NG; ++q)
              tma_load_2d(vst + q * KT * 128, &vp_map, h * D + q * 64, static_cast<int32_t>(vrow),
                          &v_full[s]);
          }
          g0 += nkt;
          if constexpr (!PERS) break;
        }
        drain_copies(v_full, issued);
      }
    } else {
      // the value rank slice of each page: lane jb < 8 resolves page jb of each tile one
      // tile ahead and issues its NG boxes, as the key copies
      constexpr int BPT = KT / kBlockSize;
      if (lane == 0) prefetch_tmap(&vp_map);
      const int32_t* table = p.block_table + static_cast<int64_t>(b) * p.bt_stride;
      const int pg0 = tile_of(0) * BPT + lane;
      int32_t nxt = (lane < BPT && nkt > 0 && page_read(pg0)) ? table[pg0] : -1;
      int issued = 0;
      for (int j = 0; j < nkt; ++j) {
        const int s = j % NS;
        const bool mine = lane < BPT && page_read(tile_of(j) * BPT + lane);
        const int32_t id = mine ? nxt : -1;
        const int32_t phys = (id >= 0 && id < p.num_blocks) ? id : -1;   // keys report bad ids
        const int nb = tile_of(j + 1) * BPT + lane;
        nxt = (lane < BPT && j + 1 < nkt && page_read(nb)) ? table[nb] : -1;
        const int nload = __popc(__ballot_sync(0xffffffffu, phys >= 0));
        bool go = true;
        if (lane == 0) {
          go = j < NS || mbar_wait(&v_empty[s], ((j / NS) - 1) & 1, abort_flag, p.dev_err);
          if (go) mbar_arrive_expect_tx(&v_full[s], nload * NG * 2048);
        }
        if (!__shfl_sync(0xffffffffu, go, 0)) break;
        issued = j + 1;
        uint8_t* vst = sm + L::ST_OFF + s * L::STAGE + L::K_BYTES;
        if (phys >= 0) {
#pragma unroll
          for (int g = 0; g < NG; ++g)
            tma_load_2d(vst + (g * BPT + lane) * 2048, &vp_map, slice * RQ + g * 64,
                        phys * kBlockSize, &v_full[s]);
        }
      }
      // the W_v rows of this slice, into stage memory once every value MMA is done
      if (lane == 0 && mbar_wait(acc_done, 0, abort_flag, p.dev_err)) {
        mbar_arrive_expect_tx(w_full, L::W_BYTES);
        uint8_t* wst = sm + L::W_OFF;
        for (int g = 0; g < D / 64; ++g)
          for (int kb = 0; kb < RQ / 64; ++kb)
            tma_load_2d(wst + (g * (RQ / 64) + kb) * 8192, &w_map, h * D + g * 64,
                        slice * RQ + kb * 64, w_full);
        mbar_wait_drain(w_full, 0);
      }
      if (lane == 0) drain_copies(v_full, issued);
    }
  } else if (warp == 1) {
    // ----------------------------------------------------------------------- MMAs
    // Issues whichever MMA is ready (non-blocking probes): the score MMA of tile js once
    // its keys landed and the softmax of tile js-2 released that S buffer, the value MMA
    // of tile jp once its weights are written and its values landed.  The tensor pipe
    // runs them in order, so S(j+1) overlaps the softmax of tile j and PV(j) overlaps
    // the softmax of tile j+1.
    if constexpr (MOD) {
      // S(0), S(1), then PV(j) and S(j + 2) in turn.  The whole warp runs the loop and one
      // elected lane issues, which leaves the descriptors in uniform registers, and the waits
      // block instead of polling: with the loop below a tile's two products took 2200 cycles
      // from weights to scores, as long as its softmax, now 1700.
      constexpr uint32_t id_s = make_idesc_f16(128, KT, false, false);
      constexpr uint32_t id_pv = make_idesc_f16(128, VN, false, true);
      const uint32_t tm = __shfl_sync(0xffffffffu, tmem, 0);
      const uint64_t qd0 = make_sdesc(smem_u32(sm), 16, 1024, kSwizzle128B);
      const uint64_t pd = make_sdesc(smem_u32(sm + L::P_OFF), 16, 1024, kSwizzle128B);
      const uint64_t kd0 = make_sdesc(smem_u32(sm + L::ST_OFF), 16, 1024, kSwizzle128B);
      const uint64_t vd0 = make_sdesc(smem_u32(sm + L::ST_OFF + L::K_BYTES),
                                      (KT / kBlockSize) * 2048, 1024, kSwizzle128B);
      int ks = 0, vs = 0;                // stages of the next keys and values
      uint32_t kph = 0, vph = 0;         // their phases
      const bool leader = elect_one();
      bool ok = true;
      int gs = 0;                        // tiles whose scores have been issued
      int js = 0, ns = PERS ? 0 : nkt;   // the next one's number in its item, the item's tiles
      int its = 0, nq = 0;               // PERS: items read, those with key tiles before this one
      bool last = !PERS;                 // PERS: no item is left
      uint32_t ends = 0;                 // PERS: an item's first (1) and last (2) tile, by tile & 1
      // the item of the next scores; false: none is left, or it is not there yet and block is
      // false (while a tile is in flight, whose values this warp has to add first: an item
      // that is late may be waiting for that tile's softmax)
      auto item = [&](bool block) {
        while (PERS && js == ns && !last) {
          uint64_t* full = &item_full[its & 1];
          const uint32_t ph = (its >> 1) & 1;
          if (!__all_sync(0xffffffffu, mbar_test_wait(full, ph))) {
            if (!block) return false;
            ok = __all_sync(0xffffffffu, mbar_wait(full, ph, abort_flag, p.dev_err));
            if (!ok) return false;
          }
          ns = __reduce_max_sync(0xffffffffu, items[(its & 1) * L::ITEM]);   // (uniform, as below)
          if (lane == 0) mbar_arrive(&item_empty[its & 1]);
          ++its;
          js = 0;
          if (ns < 0) {
            last = true;
            ns = 0;
          } else if (ns > 0) {
            ok = __all_sync(0xffffffffu, mbar_wait(nq & 1 ? q_full2 : q_full, (nq >> 1) & 1,
                                                   abort_flag, p.dev_err));
            if (!ok) return false;
          }
        }
        return js < ns;
      };
      auto scores = [&](bool block) {   // whether it issued a tile's scores
        if (!item(block)) return false;
        const int g = gs & 1, qb = PERS ? nq & 1 : 0;
        ok = __all_sync(0xffffffffu, mbar_wait(&k_full[ks], kph, abort_flag, p.dev_err));
        if (!ok) return false;
        tc_fence_after();
        const uint64_t kd = kd0 + static_cast<uint64_t>(ks * (L::STAGE >> 4));
        const uint64_t qd = qd0 + static_cast<uint64_t>(qb * (2 * L::Q_BYTES >> 4));
        if (leader) {
#pragma unroll
          for (int kk = 0; kk < 4; ++kk) {
            umma_f16(tm + g * 128, qd + kk * 2, kd + kk * 2, id_s, kk > 0 ? 1u : 0u);
            umma_f16(tm + g * 128, qd + (L::Q_BYTES >> 4) + kk * 2, kd + kk * 2, id_s, 1u);
          }
          sbad[g] = kbad[gs & 7];
          mbar_arrive(&s_full[g]);
          umma_commit(&s_full[g]);
          umma_commit(&k_empty[ks]);
          if (PERS && js + 1 == ns) umma_commit(&q_empty[qb]);
        }
        __syncwarp();
        if constexpr (PERS)
          ends = (ends & ~(3u << (2 * g))) |
                 ((js == 0 ? 1u : 0u) | (js + 1 == ns ? 2u : 0u)) << (2 * g);
        ++gs;
        if (++js == ns) ++nq;
        if (++ks == NS) {
          ks = 0;
          kph ^= 1;
        }
        return true;
      };
      if constexpr (!PERS)
        ok = __all_sync(0xffffffffu, mbar_wait(q_full, 0, abort_flag, p.dev_err));
      if (ok && scores(true)) scores(false);
      for (int g = 0; ok; ++g) {
        // nothing in flight: the next item, or the end
        if (g == gs && !scores(true)) break;
        // RECON: P buffer g & 1, each with its own barriers; rank space: one P buffer
        const int pb = RECON ? (g & 1) : 0;
        ok = mbar_wait(&v_full[vs], vph, abort_flag, p.dev_err);
        ok = mbar_wait(&p_full[pb], RECON ? (g >> 1) & 1 : g & 1, abort_flag, p.dev_err) && ok;
        ok = __all_sync(0xffffffffu, ok);
        if (!ok) break;
        tc_fence_after();
        const uint64_t vd = vd0 + static_cast<uint64_t>(vs * (L::STAGE >> 4));
        const uint32_t end = PERS ? (ends >> (2 * (g & 1))) & 3u : (g == 0 ? 1u : 0u);
        const uint32_t more = (end & 1u) ^ 1u;
        if (leader) {
#pragma unroll
          for (int k = 0; k < KT / 16; ++k) {
            if constexpr (RECON)
              umma_f16_ta(tm + 256, tm + L::P_TM + pb * (KT / 2) + k * 8, vd + k * (2048 >> 4), id_pv,
                          k > 0 ? 1u : more);
            else
              umma_f16(tm + 256, pd + (k >> 2) * (16384 >> 4) + (k & 3) * 2, vd + k * (2048 >> 4),
                       id_pv, k > 0 ? 1u : more);
          }
          umma_commit(&pv_done[pb]);
          umma_commit(&v_empty[vs]);
          if (PERS && (end & 2u)) umma_commit(acc_done);
        }
        __syncwarp();
        if (++vs == NS) {
          vs = 0;
          vph ^= 1;
        }
        // the scores' buffers of tiles up to g have been read
        while (ok && gs < g + 3 && scores(false)) {
        }
      }
      if (leader) umma_commit(PERS ? o_done : acc_done);
      mbar_wait_drain(PERS ? o_done : acc_done, 0);
    }
    if (!(MOD && RECON) && lane == 0) {
      constexpr uint32_t id_s = make_idesc_f16(128, KT, false, false);
      constexpr uint32_t id_pv = make_idesc_f16(128, VN, false, true);
      constexpr uint32_t id_o = make_idesc_f16(128, D, false, true);
      const uint32_t qa = smem_u32(sm);
      const uint32_t pa = smem_u32(sm + L::P_OFF);
      if constexpr (!MOD) {
        bool ok = mbar_wait(q_full, 0, abort_flag, p.dev_err);
        int js = 0, jp = 0;
        uint64_t t_idle = 0;
        while (ok && jp < nkt) {
          bool progress = false;
          if (js < nkt && js <= jp + 1 && mbar_test_wait(&k_full[js % NS], (js / NS) & 1)) {
            tc_fence_after();
            const uint32_t ka = smem_u32(sm + L::ST_OFF + (js % NS) * L::STAGE);
#pragma unroll
            for (int kk = 0; kk < 4; ++kk) {
              const uint64_t bd = make_sdesc(ka + kk * 32, 16, 1024, kSwizzle128B);
              umma_f16(tmem + (js & 1) * 128, make_sdesc(qa + kk * 32, 16, 1024, kSwizzle128B), bd,
                       id_s, kk > 0 ? 1u : 0u);
              umma_f16(tmem + (js & 1) * 128,
                       make_sdesc(qa + L::Q_BYTES + kk * 32, 16, 1024, kSwizzle128B), bd, id_s, 1u);
            }
            umma_commit(&s_full[js & 1]);
            umma_commit(&k_empty[js % NS]);
            ++js;
            progress = true;
          }
          // RECON: P buffer jp & 1, each with its own barriers; rank space: one P buffer
          const int pb = RECON ? (jp & 1) : 0;
          const uint32_t pph = RECON ? (jp >> 1) & 1 : jp & 1;
          if (jp < js && mbar_test_wait(&p_full[pb], pph) &&
              mbar_test_wait(&v_full[jp % NS], (jp / NS) & 1)) {
            tc_fence_after();
            const uint32_t va = smem_u32(sm + L::ST_OFF + (jp % NS) * L::STAGE + L::K_BYTES);
#pragma unroll
            for (int ks = 0; ks < KT / 16; ++ks) {
              const uint64_t bd = make_sdesc(va + ks * 2048, (KT / kBlockSize) * 2048, 1024,
                                             kSwizzle128B);
              if constexpr (RECON) {
                umma_f16_ta(tmem + 256, tmem + L::P_TM + pb * (KT / 2) + ks * 8, bd, id_pv,
                            (jp > 0 || ks > 0) ? 1u : 0u);
              } else {
                const uint64_t ad = make_sdesc(pa + (ks >> 2) * 16384 + (ks & 3) * 32, 16, 1024,
                                               kSwizzle128B);
                umma_f16(tmem + 256, ad, bd, id_pv, (jp > 0 || ks > 0) ? 1u : 0u);
              }
            }
            umma_commit(&pv_done[pb]);
            umma_commit(&v_empty[jp % NS]);
            ++jp;
            progress = true;
          }
          if (progress) {
            t_idle = 0;
          } else if (*abort_flag) {
            ok = false;
          } else if (t_idle == 0) {
            t_idle = globaltimer_ns();
          } else if (globaltimer_ns() - t_idle > kWaitLimitNs) {
            *abort_flag = 1;
            atomicOr(p.dev_err, RCP_DEVERR_TIMEOUT);
            ok = false;
          }
        }
        umma_commit(acc_done);
      }
      // up-projection of this slice: O = (z_hi + z_lo) W_v[slice rows, h*d:(h+1)*d]
      if (!RECON && mbar_wait(zq_full, 0, abort_flag, p.dev_err) &&
          mbar_wait(w_full, 0, abort_flag, p.dev_err)) {
        tc_fence_after();
        const uint32_t zh = smem_u32(sm + L::ZH_OFF), zl = smem_u32(sm + L::ZL_OFF);
        const uint32_t wa = smem_u32(sm + L::W_OFF);
#pragma unroll 1
        for (int ks = 0; ks < RQ / 16; ++ks) {
          const uint32_t koff = (ks >> 2) * 16384 + (ks & 3) * 32;
          const uint64_t bd = make_sdesc(wa + ks * 2048, (RQ / 64) * 8192, 1024, kSwizzle128B);
          umma_f16(tmem, make_sdesc(zh + koff, 16, 1024, kSwizzle128B), bd, id_o, ks > 0 ? 1u : 0u);
          umma_f16(tmem, make_sdesc(zl + koff, 16, 1024, kSwizzle128B), bd, id_o, 1u);
        }
      }
      if (!RECON) umma_commit(o_done);
      mbar_wait_drain(RECON ? acc_done : o_done, 0);
    }
  } else {
    // ----------------------------------------------- softmax (one thread per query row, or
    // MOD two: with the extra arithmetic per score one warp per scheduler set the pace)
    const int quarter = warp & 3;
    const int hf = HALVES > 1 ? (warp - 2) >> 2 : 0;    // half of the tile's keys
    constexpr int KC = KT / HALVES, VC = VN / HALVES;   // this thread's keys, value columns
    const int r = quarter * 32 + lane;                  // query row within the tile
    const uint32_t tl = tmem + (static_cast<uint32_t>(quarter * 32) << 16);
    for (int it = 0, g0 = 0;; ++it) {                   // g0: tiles of the items before
      if constexpr (PERS) {
        const bool more = take_item(it, std::true_type{});
        if (!more) break;
      }
      const int ci = i0 + r;                              // chunk row
      const bool row_ok = ci < n;
      const int pos = P0 + ci;                            // keys 0 .. pos are attended
      float m_run = -INFINITY, l_run = 0.f;
      [[maybe_unused]] RowMod rm(p, h, MOD && row_ok, row0 + r, pos, pfx);
      uint8_t* pbuf = sm + L::P_OFF;
      for (int j = 0; j < nkt; ++j) {
        const int g = g0 + j, s = g & 1;
        bool ok = mbar_wait(&s_full[s], (g >> 1) & 1, abort_flag, p.dev_err);
        ok = __all_sync(0xffffffffu, ok);
        tc_fence_after();
        const int lim = row_ok ? pos - j * KT : -1;       // columns 0 .. lim are valid
        // the whole 128-column score row: eight loads in flight, one wait
        float sv[KC];
        if (ok) {
#pragma unroll
          for (int c = 0; c < KC; c += 16)
            tmem_ld16(tl + s * 128 + hf * KC + c, *reinterpret_cast<float(*)[16]>(&sv[c]));
        }
        const int t0 = tile_of(j) * KT;                   // MOD: the tile's first key,
        const int h0 = t0 + hf * KC;                      // ... and this thread's
        uint32_t seen[KC / 32] = {};                      // MOD: keys that this row sees (edge)
        bool whole = true, edge = false;
        float shift = 0.f;                                // MOD: to be added to every score
        if constexpr (MOD) {   // while the scores are on their way
          const uint32_t bad = static_cast<uint32_t>(sbad[s]);
          whole = sees_whole(t0, bad);
          edge = !ok || !row_ok || !whole;
          if (!whole && ok && row_ok) {
#pragma unroll
            for (int k = 0; k < KC / 32; ++k)
              seen[k] = rm.seen(h0 + 32 * k, bad >> ((hf * KC + 32 * k) / kBlockSize));
          }
        }
        if (ok) tmem_wait_ld();
        if constexpr (MOD) {
          shift = modify_scores(sv, p, rm, h0, edge, seen, [&]() {
#pragma unroll
            for (int c = 0; c < KC; c += 16)
              tmem_ld16(tl + s * 128 + hf * KC + c, *reinterpret_cast<float(*)[16]>(&sv[c]));
            tmem_wait_ld();
          });
          if (!whole) {   // read back when the values are dealt with, behind the maxima's barrier
            uint32_t* cm = colm + s * 16;
#pragma unroll
            for (int k = 0; k < KC / 32; ++k) {
              const uint32_t w = __reduce_or_sync(0xffffffffu, seen[k]);
              if (lane == 0) cm[quarter * 4 + hf * (KC / 32) + k] = w;
            }
          }
        }
        const bool full_tile = MOD || __all_sync(0xffffffffu, lim >= KT - 1);   // below the diagonal
        // masked columns (diagonal tiles, rows past the chunk, a failed wait) become -inf, so
        // the max and the exponentials below need no per-element test (exp2(-inf) = 0)
        if (!MOD && (!ok || !full_tile)) {
#pragma unroll
          for (int c = 0; c < KC; ++c) sv[c] = (ok && c <= lim) ? sv[c] : -INFINITY;
        }
        // row max: four independent chains of three-input maxima
        float mx;
        {
          float m4[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll
          for (int c = 0; c < KC; c += 8) {
            m4[0] = max3f(m4[0], sv[c], sv[c + 1]);
            m4[1] = max3f(m4[1], sv[c + 2], sv[c + 3]);
            m4[2] = max3f(m4[2], sv[c + 4], sv[c + 5]);
            m4[3] = max3f(m4[3], sv[c + 6], sv[c + 7]);
          }
          mx = max3f(m4[0], m4[1], fmaxf(m4[2], m4[3]));
          if constexpr (MOD) mx += shift;
          if constexpr (HALVES > 1) {
            // the row's largest: this half's and the other's.  Every softmax warp comes past these
            // barriers for every tile, whatever its waits and masks said
            float* hm = half_max + (L::HB > 1 ? s * 256 : 0);
            if (L::HB == 1) named_bar_sync(2, 32 * NSW);   // the last tile's have been read
            hm[hf * 128 + r] = mx;
            named_bar_sync(2, 32 * NSW);
            mx = fmaxf(mx, hm[(hf ^ 1) * 128 + r]);
          }
        }
        const float m_new = (mx > m_run + kPfRescale) ? mx : m_run;
        const float alpha = (m_new == m_run) ? 1.f : fast_exp2(m_run - m_new);
        uint32_t packed[KC / 2];
        float rsum;
        {
          // rows with no valid key
          const float msub = (m_new == -INFINITY) ? 0.f : (MOD ? m_new - shift : m_new);
          const float2 msub2 = make_float2(msub, msub);
          float2 s4[4];
#pragma unroll
          for (int q = 0; q < 4; ++q) s4[q] = make_float2(0.f, 0.f);
          // the row sum is taken in fp32 before the weights are rounded to fp16; pairs of
          // columns go through the packed fp32x2 add / subtract
#pragma unroll
          for (int c = 0; c < KC; c += 2) {
            const float2 d = sub_f32x2(make_float2(sv[c], sv[c + 1]), msub2);
            const float2 pp = make_float2(fast_exp2(d.x), fast_exp2(d.y));
            s4[(c >> 1) & 3] = add_f32x2(s4[(c >> 1) & 3], pp);
            const __half2 hp = __floats2half2_rn(pp.x, pp.y);
            packed[c / 2] = *reinterpret_cast<const uint32_t*>(&hp);
          }
          const float2 t2 = add_f32x2(add_f32x2(s4[0], s4[1]), add_f32x2(s4[2], s4[3]));
          rsum = t2.x + t2.y;
        }
        // rank space: the previous tile's value MMA must be done before P is overwritten or
        // Z rescaled.  RECON: P buffer j & 1 must be free (value MMA of tile j-2), and only a
        // rescale needs the previous tile's value MMA
        const bool rescale = __any_sync(0xffffffffu, ok && alpha != 1.f && j > 0);
        if constexpr (RECON) {
          if (g >= 2)
            ok = mbar_wait(&pv_done[g & 1], ((g - 2) >> 1) & 1, abort_flag, p.dev_err) && ok;
          if (rescale)
            ok = mbar_wait(&pv_done[(g - 1) & 1], ((g - 1) >> 1) & 1, abort_flag, p.dev_err) && ok;
        } else {
          if (j > 0) ok = mbar_wait(&pv_done[0], (j - 1) & 1, abort_flag, p.dev_err) && ok;
        }
        ok = __all_sync(0xffffffffu, ok);
        tc_fence_after();
        // tcgen05.ld / st are warp-collective: the whole warp rescales when any lane needs it
        // (lanes whose max did not move multiply by 1)
        if (ok && rescale) {
#pragma unroll 1
          for (int c = hf * VC; c < (hf + 1) * VC; c += 32) {
            float v[16], w[16];
            tmem_ld16(tl + 256 + c, v);
            tmem_ld16(tl + 256 + c + 16, w);
            tmem_wait_ld();
#pragma unroll
            for (int e = 0; e < 16; ++e) {
              v[e] *= alpha;
              w[e] *= alpha;
            }
            tmem_st16(tl + 256 + c, v);
            tmem_st16(tl + 256 + c + 16, w);
          }
          tmem_wait_st();
        }
        if constexpr (RECON) {
          // P row r into tensor memory lane r: column c holds keys 2c and 2c+1
          if (ok) {
#pragma unroll
            for (int c = 0; c < KC / 2; c += 16)
              tmem_st16u(tl + L::P_TM + (g & 1) * (KT / 2) + hf * (KC / 2) + c, &packed[c]);
            tmem_wait_st();
          }
        } else {
          // P row r, K-major, 128-byte swizzle: 16-byte chunk c of the row sits at c ^ (r % 8)
#pragma unroll
          for (int ch = 0; ch < KC / 8; ++ch) {
            const int kb = (hf * (KC / 8) + ch) >> 3, cc = ch & 7;
            *reinterpret_cast<uint4*>(pbuf + kb * 16384 + r * 128 + ((cc ^ (r & 7)) << 4)) =
                make_uint4(packed[ch * 4], packed[ch * 4 + 1], packed[ch * 4 + 2],
                           packed[ch * 4 + 3]);
          }
        }
        l_run = l_run * alpha + rsum;
        m_run = m_new;
        if (MOD && !whole) {
          // keys that no row of the CTA sees (among them tokens past the end and rejected pages):
          // the same
          const uint32_t* cm = colm + s * 16;
          uint32_t unseen[4];
#pragma unroll
          for (int k = 0; k < 4; ++k) unseen[k] = ~(cm[k] | cm[4 + k] | cm[8 + k] | cm[12 + k]);
          if (unseen[0] | unseen[1] | unseen[2] | unseen[3]) {
            ok = mbar_wait(&v_full[g % NS], (g / NS) & 1, abort_flag, p.dev_err) && ok;
            zero_values(g, unseen, threadIdx.x - 64, 32 * NSW);
          }
        }
        if (!MOD && j * KT + KT > Lb) {
          // tokens past the end of the request: zero their value rows so that whatever the
          // slots hold (or stale bytes of skipped pages) never meet a zero weight as 0 * NaN
          ok = mbar_wait(&v_full[j % NS], (j / NS) & 1, abort_flag, p.dev_err) && ok;
          uint8_t* vst = sm + L::ST_OFF + (j % NS) * L::STAGE + L::K_BYTES;
          const int first = Lb - j * KT > 0 ? Lb - j * KT : 0;
          const int nrow = KT - first;
          for (int idx = threadIdx.x - 64; idx < nrow * NG * 8; idx += 128) {   // warps 2-5
            const int tok = first + idx / (NG * 8);
            const int rem = idx % (NG * 8);
            const int g = rem >> 3, ch = rem & 7;
            *reinterpret_cast<uint4*>(vst + (g * (KT / kBlockSize) + tok / kBlockSize) * 2048 +
                                      (tok % kBlockSize) * 128 + ch * 16) = make_uint4(0, 0, 0, 0);
          }
        }
        fence_proxy_async_smem();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(&p_full[RECON ? (g & 1) : 0]);
      }
      bool ok = true;
      int na = 0;                                       // PERS: items with key tiles before it
      if constexpr (PERS) {   // read again instead of holding registers through the tiles
        const int* m = items + (it & 1) * L::ITEM;
        h = m[2];
        row0 = m[3];
        i0 = m[4];
        n = m[5];
        na = m[11];
      }
      if (!PERS || nkt > 0) {
        ok = __all_sync(0xffffffffu, mbar_wait(acc_done, na & 1, abort_flag, p.dev_err));
        tc_fence_after();
        if constexpr (HALVES > 1) {   // the halves' sums (every thread is done with its last tile)
          float* hs = PERS ? half_sum : half_max;
          hs[hf * 128 + r] = l_run;
          named_bar_sync(2, 32 * NSW);
          l_run += hs[(hf ^ 1) * 128 + r];
        }
      }
      const float inv = l_run > 0.f ? 1.f / l_run : 0.f;
      if constexpr (RECON) {
        // ------------------------------------------- O / l straight to the output rows
        if (ok) {   // warp-uniform: every lane loads, only rows of the chunk are stored
          __half* dst = static_cast<__half*>(p.out) + (static_cast<size_t>(row0 + r) * H + h) * D;
          // PERS: through this item's query buffer, from which a warp stores whole 128-byte
          // pieces of rows (16-byte chunk c of a row's half at c ^ (r % HC)); a lane storing its
          // own row takes a memory access per row and chunk, 3500 cycles of the tile against 1900
          constexpr int HC = D / 8 / HALVES;               // 16-byte chunks of a half
          uint8_t* stage = sm + (na & 1) * 2 * L::Q_BYTES + quarter * 32 * D * 2 + hf * HC * 16;
#pragma unroll 1
          for (int c = hf * (D / HALVES); c < (hf + 1) * (D / HALVES); c += 16) {
            float v[16];
            __syncwarp();   // lanes past the chunk have not stored
            tmem_ld16(tl + 256 + c, v);
            tmem_wait_ld();
            uint32_t w8[8];
#pragma unroll
            for (int e = 0; e < 16; e += 2) {
              if (MOD && !(l_run > 0.f)) v[e] = v[e + 1] = 0.f;   // saw no key: no accumulator
              const __half2 hv = __floats2half2_rn(v[e] * inv, v[e + 1] * inv);
              w8[e / 2] = *reinterpret_cast<const uint32_t*>(&hv);
            }
            const uint4 w0 = make_uint4(w8[0], w8[1], w8[2], w8[3]);
            const uint4 w1 = make_uint4(w8[4], w8[5], w8[6], w8[7]);
            if (PERS && nkt > 0) {
              const int k = c / 8 - hf * HC, x = lane & (HC - 1);
              *reinterpret_cast<uint4*>(stage + lane * D * 2 + ((k ^ x) << 4)) = w0;
              *reinterpret_cast<uint4*>(stage + lane * D * 2 + (((k + 1) ^ x) << 4)) = w1;
            } else if (i0 + r < n) {
              *reinterpret_cast<uint4*>(dst + c) = w0;
              *reinterpret_cast<uint4*>(dst + c + 8) = w1;
            }
          }
          if (PERS && nkt > 0) {
            __syncwarp();
            const int k = lane % HC;
            dst = static_cast<__half*>(p.out) + (static_cast<size_t>(row0) * H + h) * D +
                  (hf * HC + k) * 8;
#pragma unroll
            for (int x0 = 0; x0 < 32; x0 += 32 / HC) {
              const int x = x0 + lane / HC, row = quarter * 32 + x;
              const uint4 w =
                  *reinterpret_cast<const uint4*>(stage + x * D * 2 + ((k ^ (x & (HC - 1))) << 4));
              if (i0 + row < n)
                *reinterpret_cast<uint4*>(dst + static_cast<size_t>(row) * H * D) = w;
            }
            fence_proxy_async_smem();   // the next queries arrive by the async proxy
            __syncwarp();
            if (lane == 0) mbar_arrive(&q_empty[na & 1]);
          }
        }
      } else {
        // ------------------------------------------- normalise z, split into fp16 hi + lo
        uint8_t* zh = sm + L::ZH_OFF;
        uint8_t* zl = sm + L::ZL_OFF;
#pragma unroll 1
        for (int c = hf * (RQ / HALVES); c < (hf + 1) * (RQ / HALVES); c += 32) {
          float v[32];
          if (ok) {
            tmem_ld16(tl + 256 + c, *reinterpret_cast<float(*)[16]>(&v[0]));
            tmem_ld16(tl + 256 + c + 16, *reinterpret_cast<float(*)[16]>(&v[16]));
            tmem_wait_ld();
          } else {
#pragma unroll
            for (int e = 0; e < 32; ++e) v[e] = 0.f;
          }
          uint32_t hw[16], lw[16];
#pragma unroll
          for (int e = 0; e < 32; e += 2) {
            if (MOD && !(l_run > 0.f)) v[e] = v[e + 1] = 0.f;   // saw no key: no accumulator
            const float z0 = v[e] * inv, z1 = v[e + 1] * inv;
            const __half2 hi = __floats2half2_rn(z0, z1);
            const float2 hb = __half22float2(hi);
            const __half2 lo = __floats2half2_rn(z0 - hb.x, z1 - hb.y);
            hw[e / 2] = *reinterpret_cast<const uint32_t*>(&hi);
            lw[e / 2] = *reinterpret_cast<const uint32_t*>(&lo);
          }
#pragma unroll
          for (int q4 = 0; q4 < 4; ++q4) {
            const int ch = (c + q4 * 8) / 8;                   // 16-byte chunk index in the row
            const int kb = ch >> 3, cc = ch & 7;
            const int off = kb * 16384 + r * 128 + ((cc ^ (r & 7)) << 4);
            *reinterpret_cast<uint4*>(zh + off) =
                make_uint4(hw[q4 * 4], hw[q4 * 4 + 1], hw[q4 * 4 + 2], hw[q4 * 4 + 3]);
            *reinterpret_cast<uint4*>(zl + off) =
                make_uint4(lw[q4 * 4], lw[q4 * 4 + 1], lw[q4 * 4 + 2], lw[q4 * 4 + 3]);
          }
        }
        fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) mbar_arrive(zq_full);
      }
      if constexpr (!PERS) break;
      __syncwarp();
      if (lane == 0) mbar_arrive(&item_empty[it & 1]);
      g0 += nkt;
    }
  }
  __syncwarp();

  // ------------------------------------------------------------------- outputs
  const bool have_o =
      RECON || __all_sync(0xffffffffu, mbar_wait(o_done, 0, abort_flag, p.dev_err));
  tc_fence_after();
  __half* out = static_cast<__half*>(p.out);
  if constexpr (RECON) {
    (void)have_o;
    (void)out;   // written by the softmax warps
  } else if constexpr (NQ == 1) {
    if (warp >= 2 && warp < 6) {
      const int r = (warp & 3) * 32 + lane;
      const uint32_t tl = tmem + (static_cast<uint32_t>((warp & 3) * 32) << 16);
      if (have_o) {   // warp-uniform: every lane loads, only rows of the chunk are stored
        __half* dst = out + (static_cast<size_t>(row0 + r) * H + h) * D;
        const bool store = i0 + r < n;
#pragma unroll 1
        for (int c = 0; c < D; c += 16) {
          float v[16];
          __syncwarp();   // lanes past the chunk have not stored
          tmem_ld16(tl + c, v);
          tmem_wait_ld();
          uint32_t w8[8];
#pragma unroll
          for (int e = 0; e < 16; e += 2) {
            const __half2 hv = __floats2half2_rn(v[e], v[e + 1]);
            w8[e / 2] = *reinterpret_cast<const uint32_t*>(&hv);
          }
          if (store) {
            *reinterpret_cast<uint4*>(dst + c) = make_uint4(w8[0], w8[1], w8[2], w8[3]);
            *reinterpret_cast<uint4*>(dst + c + 8) = make_uint4(w8[4], w8[5], w8[6], w8[7]);
          }
        }
      }
    }
  } else {
    constexpr int RPC = L::RPC;
    cluster_sync_all();                 // every slice is done reading its z hi / lo
    float* recv = reinterpret_cast<float*>(sm + L::ZH_OFF);   // [NQ][RPC][D]
    if (warp >= 2 && warp < 6) {
      const int r = (warp & 3) * 32 + lane;
      const uint32_t tl = tmem + (static_cast<uint32_t>((warp & 3) * 32) << 16);
      const uint32_t dst = map_to_rank(smem_u32(recv), static_cast<uint32_t>(r / RPC)) +
                           ((slice * RPC + r % RPC) * D) * 4;
#pragma unroll 1
      for (int c = 0; c < D; c += 16) {
        float v[16];
        if (have_o) {
          tmem_ld16(tl + c, v);
          tmem_wait_ld();
        } else {
#pragma unroll
          for (int e = 0; e < 16; ++e) v[e] = 0.f;
        }
#pragma unroll
        for (int e = 0; e < 16; e += 4) st_cluster_v4(dst + (c + e) * 4, v[e], v[e + 1], v[e + 2], v[e + 3]);
      }
    }
    cluster_sync_all();
    for (int idx = threadIdx.x; idx < RPC * D / 2; idx += W::THREADS) {
      const int rr = idx / (D / 2), d2 = (idx % (D / 2)) * 2;
      float a0 = 0.f, a1 = 0.f;
#pragma unroll
      for (int s = 0; s < NQ; ++s) {
        a0 += recv[(s * RPC + rr) * D + d2];
        a1 += recv[(s * RPC + rr) * D + d2 + 1];
      }
      const int r = slice * RPC + rr;
      if (i0 + r < n)
        *reinterpret_cast<__half2*>(out + (static_cast<size_t>(row0 + r) * H + h) * D + d2) =
            __floats2half2_rn(a0, a1);
    }
  }
  tc_fence_before();
  __syncthreads();
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc(tmem, L::TMEM_COLS);
  }
}

// --------------------------------------------------------------------------- launches
template <class S>
cudaError_t prepare_prefill() {
  auto set = [](auto kernel, int smem) {
    return cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
  };
  cudaError_t e = set(prefill_kernel<S, false, false, false>, PfSmem<S, false>::ALLOC);
  if (e == cudaSuccess) e = set(prefill_kernel<S, true, false, false>, PfSmem<S, true>::ALLOC);
  if (e == cudaSuccess)
    e = set(prefill_kernel<S, false, true, false>, PfSmem<S, false, true>::ALLOC);
  if (e == cudaSuccess) e = set(prefill_kernel<S, true, true, false>, PfSmem<S, true, true>::ALLOC);
  if (e == cudaSuccess)
    e = set(prefill_kernel<S, true, true, true>, PfSmem<S, true, true, true>::ALLOC);
  return e;
}

// recon: vp is the tensor map of V^ ([rows][H*d], 64 x 128 boxes) and w is not read.
template <class S>
cudaError_t launch_prefill(const CUtensorMap& qhi, const CUtensorMap& qlo, const CUtensorMap& kp,
                           const CUtensorMap& vp, const CUtensorMap& w, const AttnParams& p,
                           int max_tiles, int num_sms, cudaStream_t stream, bool pdl, bool recon) {
  const int NQ = recon ? 1 : PrefillCfg<S>::NQ;
  cudaLaunchConfig_t cfg{};
  cfg.stream = stream;
  cudaLaunchAttribute attr[2];
  int na = 0;
  attr[na].id = cudaLaunchAttributeClusterDimension;
  attr[na].val.clusterDim.x = NQ;
  attr[na].val.clusterDim.y = 1;
  attr[na].val.clusterDim.z = 1;
  ++na;
  if (pdl) {
    attr[na].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[na].val.programmaticStreamSerializationAllowed = 1;
    ++na;
  }
  cfg.attrs = attr;
  cfg.numAttrs = na;
  auto go = [&](auto kernel, int ctas, int threads, int smem) {
    cfg.gridDim = dim3(ctas);
    cfg.blockDim = dim3(threads);
    cfg.dynamicSmemBytes = smem;
    return cudaLaunchKernelEx(&cfg, kernel, qhi, qlo, kp, vp, w, p);
  };
  constexpr int T = PfWarps<false>::THREADS, TM = PfWarps<true>::THREADS;
  const int ctas = max_tiles * S::H * NQ;
  if (!p.mod)
    return recon ? go(prefill_kernel<S, true, false, false>, ctas, T, PfSmem<S, true>::ALLOC)
                 : go(prefill_kernel<S, false, false, false>, ctas, T, PfSmem<S, false>::ALLOC);
  if (!recon)
    return go(prefill_kernel<S, false, true, false>, ctas, TM, PfSmem<S, false, true>::ALLOC);
  // (query tile, head) items: of n rows a request has at most (n + 127) / 128 tiles.  Where every
  // item has an SM of its own, a CTA per item starts sooner (500 rows of one request behind
  // 32500 tokens 140 us against 142, 5-row chunks of four requests 53.5 against 55); with more
  // items than SMs the CTAs take them in turn (2 x 4096 above; 16 x (4096 + 256) within 1 %).
  const int64_t items = (p.nq + int64_t{127} * p.batch) / 128 * S::H;
  if (items <= num_sms)
    return go(prefill_kernel<S, true, true, false>, static_cast<int>(items), TM,
              PfSmem<S, true, true>::ALLOC);
  return go(prefill_kernel<S, true, true, true>, num_sms, TM, PfSmem<S, true, true, true>::ALLOC);
}

template cudaError_t prepare_prefill<ShapeMain>();
template cudaError_t prepare_prefill<ShapeTiny>();
template cudaError_t launch_prefill<ShapeMain>(const CUtensorMap&, const CUtensorMap&,
                                               const CUtensorMap&, const CUtensorMap&,
                                               const CUtensorMap&, const AttnParams&, int, int,
                                               cudaStream_t, bool, bool);
template cudaError_t launch_prefill<ShapeTiny>(const CUtensorMap&, const CUtensorMap&,
                                               const CUtensorMap&, const CUtensorMap&,
                                               const CUtensorMap&, const AttnParams&, int, int,
                                               cudaStream_t, bool, bool);

}  // namespace rcp
