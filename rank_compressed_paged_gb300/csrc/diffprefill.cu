// Differential attention, chunked prefill: for head pair p and query row i
//
//     x = sum_t (softmax(s_2p)_t - lam_p softmax(s_2p+1)_t) V^_p[t],   V^_p = C_v W_v[:, 2 p d : (2 p + 2) d]
//
// over the values that the reconstruction GEMM (recon.cu) rebuilt, with every score modification
// of scoremod.cuh, and the pair's 2 d outputs divided by their root mean square where a weight
// is given.
//
// The two maps have a running maximum and sum each, so their weights cannot be joined before the
// value product without a second pass over the scores.  A cluster of two CTAs takes (128 query
// rows, pair), one map each: scores and softmax are done once per head, as in prefill.cu, and each
// CTA keeps its map's product with all 2 d value columns of the pair, 256 of tensor memory's 512.
// The other 256 are two score buffers, and the weights of a tile go back into the buffer its
// scores came from (32 columns of fp16 and 32 of their rest for each half of the keys).  At the end
// each CTA gives the other its half of the columns, a copy per warp to its shared memory, and
// finishes d columns.
//
//   S  = Q~_h C_k,h^T     tcgen05, M = 128 x N = 128 keys x K = 64 (q~ as fp16 hi + lo)
//   P  = exp2(S - m)      two threads per query row, lazy rescaling
//   O += P V^_p           tcgen05, M = 128 x N = 2 d x K = 128, P from tensor memory
//
// Warps: 0 copies keys, 1 issues the MMAs (and owns the tensor memory), 2-9 softmax and epilogue
// (warp w serves tensor-memory lanes 32 (w % 4) .. + 31, half of a tile's keys each), 10 copies
// values.
//
// Roundings: V^ is stored in fp16 by the reconstruction, as for prefill.cu.  The weights, fp16 there,
// are fp16 (hi, lo) pairs here, because a difference of maps is smaller than either: the whole is off
// by 2.9e-4 of its norm, where its own rounding to fp16 makes 2.1e-4.  Single weights would make it
// 3.35e-4 and a call of 16 x (4096 + 256) take 750 us, pairs for 48 of 64 keys 3.04e-4 and 831, all
// take 870.  4-bit keys enter as codes, whose scales multiply the scores, and 4-bit values as fp16
// pairs (recon.cu).  Everything between is fp32.
//
// Bound by the products: 2560 cycles a key tile, of about 3100, with 450 between a value product's end
// and the next one's beginning (the score product that takes its weights' place is issued between
// them) and the softmax, 1950, beside them.  16 x (4096 + 256): about 460 of the call's 870 us,
// 7.2e11 operations with the pairs (34,304 key tiles of a head, 21 MFLOP each).  Waiting for keys only
// behind the value product took 16 us more, handing the halves over by stores to the other's shared
// memory 10 more.  Sending each value tile to both CTAs at once by multicast changed nothing, handing
// the maxima over ahead of need took longer (839 -> 865 us at the time).
#include <cuda.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include <cstdint>

#include "launch.h"
#include "ptx.cuh"
#include "rcp.h"
#include "scoremod.cuh"
#include "shape.h"

namespace rcp {

constexpr int kDfSoftmax = 8;                        // softmax warps
constexpr int kDfThreads = 32 * (3 + kDfSoftmax);
constexpr float kDfRescale = 8.f;   // log2 units: weights stay below 2^8 between rescales

template <class S>
struct DfSmem {
  static constexpr int KT = PrefillCfg<S>::KT, D = S::D;
  static constexpr int VN = 2 * D;                      // value columns of a pair
  static constexpr int NG = VN / 64;                    // 64-wide groups of the value tile
  static constexpr int Q_BYTES = 128 * 128;             // one [128][64] fp16 operand
  static constexpr int K_BYTES = KT * 128;
  static constexpr int V_BYTES = KT * VN * 2;
  static constexpr int STAGE = K_BYTES + V_BYTES;
  static constexpr int NS = 2;
  static constexpr int O_TM = 256;                      // accumulator columns in tensor memory
  static constexpr int TMEM_COLS = pow2_at_least(O_TM + VN, 32);
  static constexpr int ST_OFF = 2 * Q_BYTES;            // q~ hi at 0, q~ lo at Q_BYTES
  // epilogue, fp32 [8 warps][32 rows][D / 2]: the other map's part of this CTA's columns, and this
  // map's part of the other's
  static constexpr int RECV_OFF = ST_OFF;
  static constexpr int SEND_OFF = RECV_OFF + 128 * D * 4;
  static constexpr int END = ST_OFF + NS * STAGE;
  static constexpr int NBAR = 1 + 4 * NS + 7 + kDfSoftmax;
  static constexpr int BAR_OFF = END;
  static constexpr int MISC_OFF = BAR_OFF + NBAR * 8;   // tmem slot, abort flag
  // least and largest first token of the rows per warp [8], rejected pages of each key stage [8]
  // and score buffer [2], the softmax warps' column masks [2][4][4], the row halves' maxima
  // [2][2][128], sums [2][128], sums of squares [2 CTAs][2][128]
  static constexpr int MOD_OFF = MISC_OFF + 16;
  // 4-bit pages: scales of the keys of the last eight tiles
  static constexpr int KSC_OFF = (MOD_OFF + (8 + 8 + 2 + 32 + 512 + 256 + 512) * 4 + 15) / 16 * 16;
  static constexpr int TOTAL = KSC_OFF + 8 * KT * 4;
  static constexpr int ALLOC = TOTAL + 1024;
  static_assert(ALLOC <= 227 * 1024, "shared memory budget");
  static_assert(2 * 128 * D * 4 <= NS * STAGE, "exchange");
  static_assert(O_TM + VN <= 512 && S::H % 2 == 0, "tensor memory budget; heads in pairs");
};

// KSC: the pages hold the codes of 4-bit keys, whose scales (p.kscale) multiply the scores.
template <class S, bool KSC>
__global__ void __launch_bounds__(kDfThreads, 1)
    diff_prefill_kernel(const __grid_constant__ CUtensorMap qhi_map,
                        const __grid_constant__ CUtensorMap qlo_map,
                        const __grid_constant__ CUtensorMap kp_map,
                        const __grid_constant__ CUtensorMap vp_map,
                        const __grid_constant__ AttnParams p) {
  using L = DfSmem<S>;
  constexpr int KT = L::KT, NG = L::NG, VN = L::VN, D = S::D, H = S::H, NS = L::NS;
  constexpr int NSW = kDfSoftmax, BPT = KT / kBlockSize;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* sm = reinterpret_cast<uint8_t*>(
      (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~static_cast<uintptr_t>(1023));
  uint64_t* q_full = reinterpret_cast<uint64_t*>(sm + L::BAR_OFF);
  uint64_t* k_full = q_full + 1;            // [NS] keys of a stage landed
  uint64_t* v_full = k_full + NS;           // [NS] values of a stage landed
  uint64_t* k_empty = v_full + NS;          // [NS] score MMA of the stage's tile done
  uint64_t* v_empty = k_empty + NS;         // [NS] value MMA of the stage's tile done
  uint64_t* s_full = v_empty + NS;          // [2] scores of a tile in TMEM
  uint64_t* p_full = s_full + 2;            // [2] softmax weights written
  uint64_t* pv_done = p_full + 2;           // [2] value MMA of a score buffer's weights done
  uint64_t* acc_done = pv_done + 2;
  uint64_t* part_full = acc_done + 1;       // [8] a softmax warp's part from the other map
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(sm + L::MISC_OFF);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(sm + L::MISC_OFF + 4);
  int* wlo = reinterpret_cast<int*>(sm + L::MOD_OFF);       // [8]
  int* kbad = wlo + 8;                                      // [8]
  int* sbad = kbad + 8;                                     // [2]
  uint32_t* colm = reinterpret_cast<uint32_t*>(sbad + 2);   // [2][4][4]
  float* half_max = reinterpret_cast<float*>(colm + 32);    // [2][2][128]
  float* half_sum = half_max + 512;                         // [2][128]
  float* squares = half_sum + 256;                          // [2][2][128]
  float* key_scale = reinterpret_cast<float*>(sm + L::KSC_OFF);   // [8][KT]
  // by a shuffle, which tells the compiler that a warp's role is uniform
  const int warp = __shfl_sync(0xffffffffu, threadIdx.x >> 5, 0);
  const int lane = threadIdx.x & 31;

  griddep_wait();            // plan, rank-space queries and V^ are ready
  const int map = blockIdx.x & 1;                       // cluster rank: which map of the pair
  if (static_cast<int>(blockIdx.x) / H >= *p.tcount) return;   // uniform over the cluster
  const int h = blockIdx.x % H;                         // head: 2 pair + map
  const int pair = h >> 1;
  const int slot = blockIdx.x / H;
  const int b = p.tile_b[slot];
  const int i0 = p.tile_qt[slot] * 128;                 // first chunk row of this tile
  const int c0 = p.cu_chunk[b];
  const int n = p.cu_chunk[b + 1] - c0;
  const int Lb = p.seq_lens[b];
  const int P0 = Lb - n;
  int nkt = (P0 + min(n, i0 + 128) - 1 + KT) / KT;      // key tiles (causal limit)
  const int nblk = (Lb + kBlockSize - 1) / kBlockSize;
  const int row0 = c0 + i0;

  if (threadIdx.x == 0) {
    mbar_init(q_full, 1);
    for (int s = 0; s < NS; ++s) {
      mbar_init(&k_full[s], 1);
      mbar_init(&v_full[s], 1);
      mbar_init(&k_empty[s], 1);
      mbar_init(&v_empty[s], 1);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(&s_full[i], 2);             // the commit, and the MMA thread after sbad
      mbar_init(&p_full[i], NSW);
      mbar_init(&pv_done[i], 1);
    }
    mbar_init(acc_done, 1);
    for (int w = 0; w < NSW; ++w) mbar_init(&part_full[w], 1);
    *abort_flag = 0;
    fence_mbar_init();
  }
  if (warp == 1) {
    tmem_alloc(tmem_slot, L::TMEM_COLS);
    tmem_relinquish();
  }
  // the rows' first tokens, by thread; rows past the chunk do not count
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
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  // only now: the next launch's CTAs, which hold tensor memory while they wait for this one,
  // must not take this CTA's place in it
  griddep_launch();
  const uint32_t tmem = *tmem_slot;
  // tiles [0, npt) of the prefix, then lt ..
  const int32_t pfx = view_prefix(p, b, Lb);
  const int32_t lo_min = min(min(wlo[0], wlo[1]), min(wlo[2], wlo[3]));
  const int32_t lo_max = max(max(wlo[4], wlo[5]), max(wlo[6], wlo[7]));
  const int32_t npt = (pfx + KT - 1) / KT;
  const int32_t lt = max(lo_min < INT32_MAX ? lo_min / KT : nkt, npt);
  nkt = npt + max(0, nkt - lt);
  // the nearest tile first: under a bias the running maximum settles with it
  auto tile_of = [&](int j) {
    const int i = nkt - 1 - j;
    return i >= npt ? lt + (i - npt) : i;
  };
  auto page_read = [&](int x) {             // some row of the tile may see page x
    return x < nblk && (x * kBlockSize < pfx || (x + 1) * kBlockSize > lo_min);
  };
  auto sees_whole = [&](int t0) {           // every row of the CTA sees the whole tile
    return t0 + KT <= pfx || (lo_max <= t0 && t0 + KT - 1 <= P0 + i0);
  };
  // A warp whose copies may still be under way when it has nothing left to do (a wait failed
  // somewhere) stays until they are done.
  auto drain_copies = [&](uint64_t* full, int m) {
    for (int i = max(0, m - NS); i < m; ++i) mbar_wait_drain(&full[i % NS], (i / NS) & 1);
  };
  if (warp == 0) {
    // ------------------------------------------------------------------ key copies
    // lane jb < 8 resolves page jb of each tile one tile ahead and issues that page's copy;
    // lane 0 waits for the stage and arms its byte count
    if (lane == 0) {
      prefetch_tmap(&kp_map);
      mbar_arrive_expect_tx(q_full, 2 * L::Q_BYTES);
      tma_load_2d(sm, &qhi_map, h * 64, row0, q_full);
      tma_load_2d(sm + L::Q_BYTES, &qlo_map, h * 64, row0, q_full);
    }
    const int32_t* table = p.block_table + static_cast<int64_t>(b) * p.bt_stride;
    const int pg0 = tile_of(0) * BPT + lane;
    int32_t nxt = (lane < BPT && nkt > 0 && page_read(pg0)) ? table[pg0] : -1;
    int issued = 0;
    bool ok = true;
    for (int j = 0; ok && j < nkt; ++j) {
      const int s = j % NS;
      const bool mine = lane < BPT && page_read(tile_of(j) * BPT + lane);
      int32_t phys = mine ? nxt : -1;
      if (mine && (phys < 0 || phys >= p.num_blocks)) {
        atomicOr(p.dev_err, RCP_DEVERR_BAD_BLOCK);
        phys = -1;
      }
      const int nb = tile_of(j + 1) * BPT + lane;        // the next tile's page, in flight
      nxt = (lane < BPT && j + 1 < nkt && page_read(nb)) ? table[nb] : -1;
      const uint32_t rejected = __ballot_sync(0xffffffffu, mine && phys < 0);
      const int nload = __popc(__ballot_sync(0xffffffffu, phys >= 0));
      if (lane == 0) {
        ok = j < NS || mbar_wait(&k_empty[s], ((j / NS) - 1) & 1, abort_flag, p.dev_err);
        kbad[j & 7] = static_cast<int>(rejected);       // (keys run at most NS + 2 tiles ahead)
        if (ok) mbar_arrive_expect_tx(&k_full[s], nload * (KSC ? 2048 + 64 : 2048));
      }
      ok = __shfl_sync(0xffffffffu, ok, 0);             // the byte count is armed first
      if (ok) issued = j + 1;
      if (ok && phys >= 0) {
        tma_load_2d(sm + L::ST_OFF + s * L::STAGE + lane * 2048, &kp_map, 0,
                    (phys * H + h) * kBlockSize, &k_full[s]);
        if (KSC)
          bulk_g2s(key_scale + (j & 7) * KT + lane * kBlockSize,
                   p.kscale + (static_cast<int64_t>(phys) * H + h) * kBlockSize, 64, &k_full[s]);
      }
    }
    if (lane == 0) {
      drain_copies(k_full, issued);
      mbar_wait_drain(q_full, 0);
    }
  } else if (warp == 2 + NSW) {
    // ---------------------------------------------------------------- value copies
    // V^ rows of the request's tiles are contiguous: one 64-column box of 128 keys per group
    if (lane == 0) {
      prefetch_tmap(&vp_map);
      const int64_t first = p.vcum[b] * kBlockSize;
      const TileMap<S> tm(p.vmap + 2 * b, nblk);
      const int tile0 = tm.lt - tm.np;                  // tiles that are not in V^
      int issued = 0;
      for (int j = 0; j < nkt; ++j) {
        const int s = j % NS;
        uint8_t* vst = sm + L::ST_OFF + s * L::STAGE + L::K_BYTES;
        if (j >= NS && !mbar_wait(&v_empty[s], ((j / NS) - 1) & 1, abort_flag, p.dev_err)) break;
        mbar_arrive_expect_tx(&v_full[s], L::V_BYTES);
        issued = j + 1;
        const int x = tile_of(j);
        const int64_t vrow = first + static_cast<int64_t>(x >= npt ? x - tile0 : x) * KT;
#pragma unroll
        for (int q = 0; q < NG; ++q)
          tma_load_2d(vst + q * KT * 128, &vp_map, pair * VN + q * 64, static_cast<int32_t>(vrow),
                      &v_full[s]);
      }
      drain_copies(v_full, issued);
    }
  } else if (warp == 1) {
    // ----------------------------------------------------------------------- MMAs
    // S(0), S(1), then PV(j) and, once that has read the weights out of score buffer j & 1,
    // S(j + 2) into it, while the softmax is at tile j + 1.  The whole warp runs the loop and one
    // elected lane issues, which leaves the descriptors in uniform registers.
    constexpr uint32_t id_s = make_idesc_f16(128, KT, false, false);
    constexpr uint32_t id_pv = make_idesc_f16(128, VN, false, true);
    const uint32_t tm = __shfl_sync(0xffffffffu, tmem, 0);
    const uint64_t qd = make_sdesc(smem_u32(sm), 16, 1024, kSwizzle128B);
    const uint64_t kd0 = make_sdesc(smem_u32(sm + L::ST_OFF), 16, 1024, kSwizzle128B);
    const uint64_t vd0 = make_sdesc(smem_u32(sm + L::ST_OFF + L::K_BYTES), BPT * 2048, 1024,
                                    kSwizzle128B);
    const bool leader = elect_one();
    // what a score product needs beside its buffer: the keys, and word of their rejected pages
    auto ready = [&](int j) {
      if (!__all_sync(0xffffffffu, mbar_wait(&k_full[j % NS], (j / NS) & 1, abort_flag, p.dev_err)))
        return false;
      if (leader) {
        sbad[j & 1] = kbad[j & 7];
        mbar_arrive(&s_full[j & 1]);
      }
      return true;
    };
    auto scores = [&](int j) {
      tc_fence_after();
      const uint64_t kd = kd0 + static_cast<uint64_t>((j % NS) * (L::STAGE >> 4));
      const uint32_t d = tm + (j & 1) * 128;
      if (leader) {
#pragma unroll
        for (int kk = 0; kk < 4; ++kk) {
          umma_f16(d, qd + kk * 2, kd + kk * 2, id_s, kk > 0 ? 1u : 0u);
          umma_f16(d, qd + (L::Q_BYTES >> 4) + kk * 2, kd + kk * 2, id_s, 1u);
        }
        umma_commit(&s_full[j & 1]);
        umma_commit(&k_empty[j % NS]);
      }
      __syncwarp();
    };
    bool ok = __all_sync(0xffffffffu, mbar_wait(q_full, 0, abort_flag, p.dev_err));
    for (int j = 0; ok && j < 2 && j < nkt; ++j) {
      ok = ready(j);
      if (ok) scores(j);
    }
    for (int j = 0; ok && j < nkt; ++j) {
      const int s = j % NS;
      ok = mbar_wait(&v_full[s], (j / NS) & 1, abort_flag, p.dev_err);
      ok = mbar_wait(&p_full[j & 1], (j >> 1) & 1, abort_flag, p.dev_err) && ok;
      ok = __all_sync(0xffffffffu, ok);
      if (!ok) break;
      tc_fence_after();
      const uint64_t vd = vd0 + static_cast<uint64_t>(s * (L::STAGE >> 4));
      if (leader) {
#pragma unroll
        for (int k = 0; k < KT / 16; ++k) {
          // weights of keys 0..63 at column 0, 64..127 at 64, their lo at 32 and 96
          const uint32_t pk = tm + (j & 1) * 128 + (k >> 2) * 64 + (k & 3) * 8;
          umma_f16_ta(tm + L::O_TM, pk, vd + k * (2048 >> 4), id_pv, (j > 0 || k > 0) ? 1u : 0u);
          umma_f16_ta(tm + L::O_TM, pk + 32, vd + k * (2048 >> 4), id_pv, 1u);
        }
        umma_commit(&pv_done[j & 1]);
        umma_commit(&v_empty[s]);
      }
      __syncwarp();
      if (j + 2 < nkt) {
        ok = ready(j + 2);   // (while the products run)
        ok = __all_sync(0xffffffffu, ok && mbar_wait(&pv_done[j & 1], (j >> 1) & 1, abort_flag,
                                                     p.dev_err));
        if (ok) scores(j + 2);
      }
    }
    if (leader) umma_commit(acc_done);
    mbar_wait_drain(acc_done, 0);
  }

  // ------------------------------------- softmax and epilogue (two threads per query row)
  // The other warps come along for the cluster's barriers.
  const bool soft = warp >= 2 && warp < 2 + NSW;
  const int quarter = warp & 3;
  const int hf = soft ? (warp - 2) >> 2 : 0;          // half of the tile's keys, of the columns
  constexpr int KC = KT / 2, VC = VN / 2;             // this thread's keys, value columns
  const int r = quarter * 32 + lane;                  // query row within the tile
  const uint32_t tl = tmem + (static_cast<uint32_t>(quarter * 32) << 16);
  const bool row_ok = i0 + r < n;
  float l_run = 0.f;
  bool done = true;
  if (soft) {
    const int pos = P0 + i0 + r;                      // keys 0 .. pos are attended
    float m_run = -INFINITY;
    RowMod rm(p, h, row_ok, row0 + r, pos, pfx);
    for (int j = 0; j < nkt; ++j) {
      const int s = j & 1;
      bool ok = mbar_wait(&s_full[s], (j >> 1) & 1, abort_flag, p.dev_err);
      ok = __all_sync(0xffffffffu, ok);
      tc_fence_after();
      float sv[KC];
      if (ok) {
#pragma unroll
        for (int c = 0; c < KC; c += 16)
          tmem_ld16(tl + s * 128 + hf * KC + c, *reinterpret_cast<float(*)[16]>(&sv[c]));
      }
      auto scaled = [&]() {
        if constexpr (KSC) {
          const float4* ks = reinterpret_cast<const float4*>(key_scale + (j & 7) * KT + hf * KC);
#pragma unroll
          for (int c = 0; c < KC; c += 4) {
            const float4 k4 = ks[c / 4];
            sv[c] *= k4.x;
            sv[c + 1] *= k4.y;
            sv[c + 2] *= k4.z;
            sv[c + 3] *= k4.w;
          }
        }
      };
      const int t0 = tile_of(j) * KT;                 // the tile's first key,
      const int h0 = t0 + hf * KC;                    // ... and this thread's
      uint32_t seen[KC / 32] = {};                    // keys that this row sees (edge)
      const uint32_t bad = static_cast<uint32_t>(sbad[s]);
      const bool whole = sees_whole(t0);
      const bool edge = !ok || !row_ok || !whole || bad != 0;
      if ((!whole || bad != 0) && ok && row_ok) {
#pragma unroll
        for (int k = 0; k < KC / 32; ++k)
          seen[k] = rm.seen(h0 + 32 * k, bad >> ((hf * KC + 32 * k) / kBlockSize));
      }
      if (ok) {
        tmem_wait_ld();
        scaled();
      }
      const float shift = modify_scores(sv, p, rm, h0, edge, seen, [&]() {
#pragma unroll
        for (int c = 0; c < KC; c += 16)
          tmem_ld16(tl + s * 128 + hf * KC + c, *reinterpret_cast<float(*)[16]>(&sv[c]));
        tmem_wait_ld();
        scaled();
      });
      if (!whole) {   // read back when the values are dealt with
#pragma unroll
        for (int k = 0; k < KC / 32; ++k) {
          const uint32_t w = __reduce_or_sync(0xffffffffu, seen[k]);
          if (lane == 0) colm[s * 16 + quarter * 4 + hf * (KC / 32) + k] = w;
        }
      }
      // the row's largest: this half's and the other's, from the two warps of its lanes, which come
      // past this barrier for every tile, whatever their waits and masks said
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
        mx = max3f(m4[0], m4[1], fmaxf(m4[2], m4[3])) + shift;
      }
      float* hm = half_max + s * 256;
      hm[hf * 128 + r] = mx;
      named_bar_sync(1 + quarter, 64);
      mx = fmaxf(mx, hm[(hf ^ 1) * 128 + r]);
      const float m_new = (mx > m_run + kDfRescale) ? mx : m_run;
      const float alpha = (m_new == m_run) ? 1.f : fast_exp2(m_run - m_new);
      // the weights, over this half's own scores: 32 columns of hi (column c holds keys 2c and
      // 2c + 1), then those of lo
      float rsum;
      {
        const float msub = (m_new == -INFINITY) ? 0.f : m_new - shift;   // (no valid key yet)
        const float2 msub2 = make_float2(msub, msub);
        float2 s4[4];
#pragma unroll
        for (int q = 0; q < 4; ++q) s4[q] = make_float2(0.f, 0.f);
#pragma unroll
        for (int c0 = 0; c0 < KC; c0 += 32) {
          uint32_t hi[16], lo[16];
#pragma unroll
          for (int c = 0; c < 32; c += 2) {
            const float2 d = sub_f32x2(make_float2(sv[c0 + c], sv[c0 + c + 1]), msub2);
            const float2 pp = make_float2(fast_exp2(d.x), fast_exp2(d.y));
            s4[(c >> 1) & 3] = add_f32x2(s4[(c >> 1) & 3], pp);
            const __half2 hp = __floats2half2_rn(pp.x, pp.y);
            hi[c / 2] = *reinterpret_cast<const uint32_t*>(&hp);
            const float2 lp = sub_f32x2(pp, __half22float2(hp));
            const __half2 hl = __floats2half2_rn(lp.x, lp.y);
            lo[c / 2] = *reinterpret_cast<const uint32_t*>(&hl);
          }
          if (ok) {
            tmem_st16u(tl + s * 128 + hf * 64 + c0 / 2, hi);
            tmem_st16u(tl + s * 128 + hf * 64 + 32 + c0 / 2, lo);
          }
        }
        const float2 t2 = add_f32x2(add_f32x2(s4[0], s4[1]), add_f32x2(s4[2], s4[3]));
        rsum = t2.x + t2.y;
      }
      // only a rescale needs the previous tile's value MMA
      const bool rescale = __any_sync(0xffffffffu, ok && alpha != 1.f && j > 0);
      if (rescale)
        ok = mbar_wait(&pv_done[(j - 1) & 1], ((j - 1) >> 1) & 1, abort_flag, p.dev_err) && ok;
      ok = __all_sync(0xffffffffu, ok);
      tc_fence_after();
      // tcgen05.ld / st are warp-collective: the whole warp rescales when any lane needs it
      if (ok && rescale) {
#pragma unroll 1
        for (int c = hf * VC; c < (hf + 1) * VC; c += 32) {
          float v[16], w[16];
          tmem_ld16(tl + L::O_TM + c, v);
          tmem_ld16(tl + L::O_TM + c + 16, w);
          tmem_wait_ld();
#pragma unroll
          for (int e = 0; e < 16; ++e) {
            v[e] *= alpha;
            w[e] *= alpha;
          }
          tmem_st16(tl + L::O_TM + c, v);
          tmem_st16(tl + L::O_TM + c + 16, w);
        }
      }
      tmem_wait_st();
      l_run = l_run * alpha + rsum;
      m_run = m_new;
      if (!whole) {   // (the same tiles in every warp, whatever its waits said)
        // keys that no row of the CTA sees, among them tokens past the end: their value rows become
        // zero, because 0 times what a slot holds may be NaN (those of rejected pages are zero)
        named_bar_sync(5, 32 * NSW);   // every warp's column masks are written
        const uint32_t* cm = colm + s * 16;
        uint32_t unseen[4];
#pragma unroll
        for (int k = 0; k < 4; ++k) unseen[k] = ~(cm[k] | cm[4 + k] | cm[8 + k] | cm[12 + k]);
        if (unseen[0] | unseen[1] | unseen[2] | unseen[3]) {
          mbar_wait(&v_full[j % NS], (j / NS) & 1, abort_flag, p.dev_err);
          uint8_t* vst = sm + L::ST_OFF + (j % NS) * L::STAGE + L::K_BYTES;
          for (int idx = threadIdx.x - 64; idx < KT * NG * 8; idx += 32 * NSW) {
            const int tok = idx / (NG * 8);
            const uint32_t w = tok < 64 ? (tok < 32 ? unseen[0] : unseen[1])
                                        : (tok < 96 ? unseen[2] : unseen[3]);
            if (!((w >> (tok & 31)) & 1u)) continue;
            const int rem = idx % (NG * 8), box = rem >> 3, ch = rem & 7;
            *reinterpret_cast<uint4*>(vst + (box * BPT + tok / kBlockSize) * 2048 +
                                      (tok % kBlockSize) * 128 + ch * 16) = make_uint4(0, 0, 0, 0);
          }
          fence_proxy_async_smem();    // generic stores -> the value MMA's async-proxy reads
        }
      }
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(&p_full[s]);
    }
    done = __all_sync(0xffffffffu, mbar_wait(acc_done, 0, abort_flag, p.dev_err));
    tc_fence_after();
    half_sum[hf * 128 + r] = l_run;
    named_bar_sync(1 + quarter, 64);
    l_run += half_sum[(hf ^ 1) * 128 + r];
  }
  // this map's factor: 1 / l, the second map's times -lam; a row that saw no key gives zeros
  // (there may be no accumulator)
  const bool any = l_run > 0.f && done;
  const float scale = any ? (map ? -p.lam[pair] : 1.f) / l_run : 0.f;
  constexpr int DC = D / 2, CH = DC / 4;              // this thread's columns of either half
  constexpr int PART = 32 * DC * 4;                   // bytes of a warp's part
  // 16-byte chunk c of the warp's row `lane`, among its part
  auto part_at = [&](int c) { return (lane * CH + (c ^ (lane & (CH - 1)))) * 16; };
  const int w = soft ? warp - 2 : 0;
  uint8_t* send = sm + L::SEND_OFF + w * PART;
  if (soft) {
    // the columns that the other CTA finishes (its stages are done: so are its copies and MMAs)
    if (lane == 0) mbar_arrive_expect_tx(&part_full[w], PART);
#pragma unroll 1
    for (int c = 0; c < DC; c += 16) {
      float v[16];
      __syncwarp();
      tmem_ld16(tl + L::O_TM + (map ^ 1) * D + hf * DC + c, v);
      tmem_wait_ld();
#pragma unroll
      for (int e = 0; e < 16; e += 4)
        *reinterpret_cast<float4*>(send + part_at((c + e) / 4)) =
            make_float4(any ? v[e] * scale : 0.f, any ? v[e + 1] * scale : 0.f,
                        any ? v[e + 2] * scale : 0.f, any ? v[e + 3] * scale : 0.f);
    }
    fence_proxy_async_smem();   // generic stores -> the copy's async-proxy reads
  }
  cluster_sync_all();           // both CTAs are done with their stages
  float x[DC];
  float ss = 0.f;
  if (soft) {
    const uint8_t* recv = sm + L::RECV_OFF + w * PART;
    if (lane == 0) {
      const uint32_t other = static_cast<uint32_t>(map ^ 1);
      bulk_s2peer(map_to_rank(smem_u32(recv), other), send, PART, map_to_rank(smem_u32(&part_full[w]), other));
    }
    __syncwarp();
    // meanwhile this map's part of this CTA's columns
#pragma unroll
    for (int c = 0; c < DC; c += 16) {
      tmem_ld16(tl + L::O_TM + map * D + hf * DC + c, *reinterpret_cast<float(*)[16]>(&x[c]));
      tmem_wait_ld();
#pragma unroll
      for (int e = 0; e < 16; ++e) x[c + e] = any ? x[c + e] * scale : 0.f;
    }
    const bool came = mbar_wait(&part_full[w], 0, abort_flag, p.dev_err);
#pragma unroll
    for (int c = 0; c < DC; c += 4) {
      const float4 o = came ? *reinterpret_cast<const float4*>(recv + part_at(c / 4))
                            : make_float4(0.f, 0.f, 0.f, 0.f);
      x[c] += o.x;
      x[c + 1] += o.y;
      x[c + 2] += o.z;
      x[c + 3] += o.w;
    }
    if (p.norm) {
#pragma unroll
      for (int c = 0; c < DC; ++c) ss = fmaf(x[c], x[c], ss);
      squares[(map * 2 + hf) * 128 + r] = ss;
      st_cluster_f32(map_to_rank(smem_u32(squares + (map * 2 + hf) * 128 + r),
                                 static_cast<uint32_t>(map ^ 1)), ss);
    }
  }
  cluster_sync_all();           // squares and parts are there: no CTA leaves before its part has
  if (soft && row_ok) {
    float f = p.out_scale;
    if (p.norm) {
      const float t = (squares[r] + squares[128 + r]) + (squares[256 + r] + squares[384 + r]);
      const float mean = t / VN + p.eps;               // (0: zeros stay zeros)
      f *= mean == 0.f ? 0.f : rsqrtf(mean);
    }
    __half* dst = static_cast<__half*>(p.out) + (static_cast<size_t>(row0 + r) * H + h) * D + hf * DC;
#pragma unroll
    for (int c = 0; c < DC; c += 8) {
      uint32_t w[4];
#pragma unroll
      for (int e = 0; e < 8; e += 2) {
        float a = x[c + e] * f, bb = x[c + e + 1] * f;
        if (p.norm) {
          const float2 g = __ldg(reinterpret_cast<const float2*>(p.norm + map * D + hf * DC + c + e));
          a *= g.x;
          bb *= g.y;
        }
        const __half2 hv = __floats2half2_rn(a, bb);
        w[e / 2] = *reinterpret_cast<const uint32_t*>(&hv);
      }
      *reinterpret_cast<uint4*>(dst + c) = make_uint4(w[0], w[1], w[2], w[3]);
    }
  }
  __syncwarp();
  tc_fence_before();
  __syncthreads();
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc(tmem, L::TMEM_COLS);
  }
}

template <class S>
cudaError_t prepare_diff_prefill() {
  cudaError_t e = cudaFuncSetAttribute(diff_prefill_kernel<S, false>,
                                       cudaFuncAttributeMaxDynamicSharedMemorySize, DfSmem<S>::ALLOC);
  if (e == cudaSuccess)
    e = cudaFuncSetAttribute(diff_prefill_kernel<S, true>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                             DfSmem<S>::ALLOC);
  return e;
}

template <class S>
cudaError_t launch_diff_prefill(const CUtensorMap& qhi, const CUtensorMap& qlo,
                                const CUtensorMap& kp, const CUtensorMap& vhat, const AttnParams& p,
                                cudaStream_t stream, bool pdl) {
  cudaLaunchConfig_t cfg{};
  cfg.stream = stream;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = 2;
  attr[0].val.clusterDim.y = 1;
  attr[0].val.clusterDim.z = 1;
  attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[1].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = pdl ? 2 : 1;
  // of n rows a request has at most (n + 127) / 128 tiles
  cfg.gridDim = dim3(static_cast<unsigned>((p.nq + int64_t{127} * p.batch) / 128 * S::H));
  cfg.blockDim = dim3(kDfThreads);
  cfg.dynamicSmemBytes = DfSmem<S>::ALLOC;
  if (p.kscale != nullptr)
    return cudaLaunchKernelEx(&cfg, diff_prefill_kernel<S, true>, qhi, qlo, kp, vhat, p);
  return cudaLaunchKernelEx(&cfg, diff_prefill_kernel<S, false>, qhi, qlo, kp, vhat, p);
}

template cudaError_t prepare_diff_prefill<ShapeMain>();
template cudaError_t prepare_diff_prefill<ShapeTiny>();
template cudaError_t launch_diff_prefill<ShapeMain>(const CUtensorMap&, const CUtensorMap&,
                                                    const CUtensorMap&, const CUtensorMap&,
                                                    const AttnParams&, cudaStream_t, bool);
template cudaError_t launch_diff_prefill<ShapeTiny>(const CUtensorMap&, const CUtensorMap&,
                                                    const CUtensorMap&, const CUtensorMap&,
                                                    const AttnParams&, cudaStream_t, bool);

}  // namespace rcp
