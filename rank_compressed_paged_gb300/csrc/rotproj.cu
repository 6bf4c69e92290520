// Rotated projections of many rows: key and query jobs of more than 192 tokens whose positions are
// rotated (rcp_rotary); gemm.cu has the smaller ones, and the values.
//
//     C_h = rot(X_h) U_k,h^T      X_h [rows][d] the keys (or queries) of head h, U_k,h [r_k][d]
//
// A CTA takes 128 rows and a group of HG heads (two to eight).  The angles are the same for
// every head: a thread has a row and keeps those of its slots (eight pairs each) in registers, and a
// pipeline runs over the heads: copies of X_h and U_k,h to shared memory, the rotation from there to
// tensor memory (fp32, the result an fp16 (hi, lo) pair), the product on tcgen05 (M = 128 rows from
// tensor memory, N = r_k, K = d, hi and lo), and the epilogue, where a thread holds a whole row of the
// page (all r_k ranks of its token and head), which leaves as one run, through shared memory.  Four
// stages of X and U, two operands and two accumulators.
//
// Warps: 0-15 rotate (warp w: rows 32 (w % 4) .., every fourth slot), 16-23 epilogue (lane = row;
// four warps take the even heads, four the odd ones), 24 copies, 25 MMAs and tensor memory.
//
// It runs behind the values' launch (gemm.cu), whose 64 pairs of CTAs for 4096 tokens leave 24 SMs:
// it starts there at once, without waiting for that launch (it touches nothing that launch does),
// and CTA 0 waits at its end, so that what comes behind this launch finds both complete.
//
// An append of 4096 tokens takes 45.1 us: the values alone 29.5, this kernel alone 20.4, of which 13
// are left without the rotation, the stores and the way to HBM: launch, angles, and eight heads
// one after another (832 threads have 72 registers each: at the main shape 232 bytes of a thread's
// are spilled), whose steps (rotation, products, epilogue) each take 1 to 1.5 us of an SM's
// issue, shared and tensor memory.  As jobs of gemm.cu, which rotate for two heads at a time, the
// call took 68; rotating in shared memory, with eight warps and angles read slot after slot, 47.4 (the
// rotation wrote 64 KB a head there, which the products read again).  How many heads a CTA takes is
// chosen so that the SMs behind the values' are filled (api.cu): 4096 tokens 45.9 by eight, 45.1 by
// five groups, 50.9 by four heads and 57.5 by sixteen; 2560 tokens 37.0 by eight, 29.6 by seven groups.
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

constexpr int kRpRotate = 16, kRpStore = 8, kRpThreads = 32 * (kRpRotate + kRpStore + 2);

template <class S>
struct RpSmem {
  static constexpr int KB = S::D / 64;                   // 64-wide k-blocks of a head
  static constexpr int X_BYTES = KB * 128 * 128;
  static constexpr int U_BYTES = KB * 64 * 128;
  static constexpr int STAGE = X_BYTES + U_BYTES;
  static constexpr int NS = 4;                           // stages of X and U
  static constexpr int OUT_OFF = NS * STAGE;             // results of an epilogue warp, [kRpStore]
  static constexpr int OUT_BYTES = 32 * 128;
  static constexpr int BAR_OFF = OUT_OFF + kRpStore * OUT_BYTES;   // full, empty [NS], turned, acc, drained [2]
  static constexpr int MISC_OFF = BAR_OFF + (2 * NS + 6) * 8;   // tmem slot, abort flag
  static constexpr int TOTAL = MISC_OFF + 16;
  static constexpr int ALLOC = TOTAL + 1024;
  // tensor memory: two accumulators, 64 columns apart, then two operands of D / 2 columns hi and as
  // many lo
  static constexpr int A_TM = 128;
  static constexpr int TMEM_COLS = pow2_at_least(A_TM + 2 * S::D, 32);
  static_assert(kRpStore * OUT_BYTES >= 128 * 2 * S::D, "half of the angles are staged there");
  static_assert(S::RK % 16 == 0 && S::RK <= 64 && S::D % 64 == 0, "shape");
  static_assert(A_TM + 2 * S::D <= 512 && ALLOC <= 227 * 1024, "tensor and shared memory budget");
};

// Stores a warp's 32 rows of PCS 16-byte pieces (this lane's row: w, to dst, or nowhere) as whole
// runs: through `stage`, from which neighbouring lanes take a row's neighbouring pieces.
template <int PCS>
__device__ __forceinline__ void store_rows(uint8_t* stage, int lane, const uint4 (&w)[PCS],
                                           uint8_t* dst) {
#pragma unroll
  for (int c = 0; c < PCS; ++c)
    *reinterpret_cast<uint4*>(stage + (lane * PCS + (c ^ (lane & (PCS - 1)))) * 16) = w[c];
  __syncwarp();
#pragma unroll
  for (int k = 0; k < PCS; ++k) {
    const int i = k * 32 + lane, row = i / PCS, c = i % PCS;
    uint8_t* to = reinterpret_cast<uint8_t*>(
        __shfl_sync(0xffffffffu, reinterpret_cast<unsigned long long>(dst), row));
    const uint4 v = *reinterpret_cast<const uint4*>(stage + (row * PCS + (c ^ (row & (PCS - 1)))) * 16);
    if (to != nullptr) *reinterpret_cast<uint4*>(to + c * 16) = v;
  }
  __syncwarp();
}

template <class S>
__global__ void __launch_bounds__(kRpThreads, 1)
    rotated_proj_kernel(const __grid_constant__ CUtensorMap u_map,
                        const __grid_constant__ CUtensorMap k_map,
                        const __grid_constant__ CUtensorMap q_map, const AppendParams p,
                        int key_tiles, int behind_values) {
  using L = RpSmem<S>;
  constexpr int KB = L::KB, D = S::D, RK = S::RK, NS = L::NS;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* sm = reinterpret_cast<uint8_t*>(
      (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~static_cast<uintptr_t>(1023));
  uint64_t* full = reinterpret_cast<uint64_t*>(sm + L::BAR_OFF);   // [NS] X and U landed
  uint64_t* empty = full + NS;                                     // [NS] the stage's MMAs done
  uint64_t* turned = empty + NS;                                   // [2] rotated (kRpRotate warps)
  uint64_t* acc = turned + 2;                                      // [2] MMAs done
  uint64_t* drained = acc + 2;                                     // [2] accumulator read (4 warps)
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(sm + L::MISC_OFF);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(sm + L::MISC_OFF + 4);
  // by a shuffle, which tells the compiler that a warp's role is uniform
  const int warp = __shfl_sync(0xffffffffu, threadIdx.x >> 5, 0), lane = threadIdx.x & 31;
  const int groups = p.proj_groups, grp = blockIdx.x % groups, tile = blockIdx.x / groups;
  const int h0 = grp * S::H / groups, HG = (grp + 1) * S::H / groups - h0;   // this CTA's heads
  const bool query = tile >= key_tiles;
  const int n0 = (query ? tile - key_tiles : tile) * 128;
  const int n = query ? p.nq : p.T;
  const int32_t* pos = query ? p.q_pos : p.k_pos;

  if (threadIdx.x == 0) {
    for (int i = 0; i < NS; ++i) {
      mbar_init(&full[i], 1);
      mbar_init(&empty[i], 1);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(&turned[i], kRpRotate);
      mbar_init(&acc[i], 1);
      mbar_init(&drained[i], 4);
    }
    *abort_flag = 0;
    fence_mbar_init();
  }
  if (warp == kRpRotate + kRpStore + 1) {
    tmem_alloc(tmem_slot, L::TMEM_COLS);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;
  // behind the values' launch everything before that one is complete; else this one waits, at its
  // end where the launch ahead writes nothing that it touches
  if (!behind_values && !p.wait_at_exit) griddep_wait();
  griddep_launch();

  if (warp < kRpRotate) {
    // ------------------------------------------------------------------------- rotation
    // slot t of a row: pairs 8 t .. 8 t + 7, in chunks (of eight elements) t and t + units, or
    // (interleaved) 2 t and 2 t + 1; behind the pairs, chunks 2 t and 2 t + 1 as they are
    constexpr int SLOTS = D / 64;                         // of this thread: every fourth
    const int units = pos ? p.rot_dim / 16 : 0, half = p.rot_dim / 2;
    const int r = (warp & 3) * 32 + lane, t0 = warp >> 2;
    const uint32_t at = pos && n0 + r < n ? static_cast<uint32_t>(pos[n0 + r]) : 0u;
    const bool in = at < static_cast<uint32_t>(p.num_pos);
    const bool zero = pos && query && !in;                // (a key without a position is not stored)
    if (zero && t0 == 0) atomicOr(p.dev_err, RCP_DEVERR_BAD_POS);
    // the angles: a warp reads eight rows of the table, whole (row 0 for rows without a position);
    // cosines, then sines, go through shared memory to the threads that keep them
    float cs[SLOTS][8], sn[SLOTS][8];
    float far = 1.f;                                      // most that a rotation lengthens by
    if (units > 0) {
      float4 ang[8];
      const int pcs = half / 4;
#pragma unroll
      for (int k = 0; k < 8; ++k) {
        const int row = warp * 8 + k;
        uint32_t to = n0 + row < n ? static_cast<uint32_t>(pos[n0 + row]) : 0u;
        if (to >= static_cast<uint32_t>(p.num_pos)) to = 0;
        if (lane < 2 * pcs)
          ang[k] = __ldg(reinterpret_cast<const float4*>(p.rot_table + static_cast<int64_t>(to) * p.rot_dim) + lane);
      }
      uint8_t* st = sm + L::OUT_OFF;
#pragma unroll
      for (int part = 0; part < 2; ++part) {
        const int c = lane - part * pcs;
        if (part == 1) named_bar_sync(1, 32 * kRpRotate);
        if (c >= 0 && c < pcs)
#pragma unroll
          for (int k = 0; k < 8; ++k) {
            const int row = warp * 8 + k;
            *reinterpret_cast<float4*>(st + row * 2 * D + ((c ^ row) & (D / 8 - 1)) * 16) = ang[k];
          }
        named_bar_sync(1, 32 * kRpRotate);
#pragma unroll
        for (int k = 0; k < SLOTS; ++k) {
          const int t = t0 + 4 * k;
          if (t >= units) continue;
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            const float4 v = *reinterpret_cast<const float4*>(
                st + r * 2 * D + (((2 * t + e) ^ r) & (D / 8 - 1)) * 16);
            float* to = part ? sn[k] : cs[k];
            to[4 * e] = v.x; to[4 * e + 1] = v.y; to[4 * e + 2] = v.z; to[4 * e + 3] = v.w;
          }
        }
      }
    }
#pragma unroll
    for (int k = 0; k < SLOTS; ++k)
      if (t0 + 4 * k < units)
#pragma unroll
        for (int e = 0; e < 8; ++e) far = fmaxf(far, fabsf(cs[k][e]) + fabsf(sn[k][e]));
    // elements below this stay within fp16 (a table may hold more than cosines and sines)
    const __half2 near = __half2half2(__float2half_rd(65000.f / far));
    const uint32_t trow = tmem + (static_cast<uint32_t>((warp & 3) * 32) << 16) + L::A_TM;
    auto chunk = [&](int c) {   // byte offset of the row's 16-byte chunk c
      return (c >> 3) * (128 * 128) + r * 128 + (((c & 7) ^ (r & 7)) << 4);
    };
    for (int i = 0; i < HG; ++i) {
      const int s = i & 1;
      const uint8_t* x = sm + (i % NS) * L::STAGE;
      bool ok = mbar_wait(&full[i % NS], (i / NS) & 1, abort_flag, p.dev_err);
      if (i >= 2)   // head i - 2's products have read the operand
        ok = mbar_wait(&acc[s], ((i >> 1) - 1) & 1, abort_flag, p.dev_err) && ok;
      ok = __all_sync(0xffffffffu, ok);
      tc_fence_after();
      const uint32_t hi_tm = trow + s * D, lo_tm = hi_tm + D / 2;
#pragma unroll
      for (int k = 0; k < SLOTS; ++k) {
        const int t = t0 + 4 * k;
        const bool turn = t < units, apart = turn && !p.interleaved;
        const int c0 = apart ? t : 2 * t, c1 = apart ? t + units : 2 * t + 1;
        const uint4 a = *reinterpret_cast<const uint4*>(x + chunk(c0));
        const uint4 b = *reinterpret_cast<const uint4*>(x + chunk(c1));
        uint32_t hw[8] = {a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w}, lw[8] = {};
        if (turn) {
          float2 f[8];
          __half2 big = __float2half2_rn(0.f);   // largest magnitude, NaN kept
#pragma unroll
          for (int e = 0; e < 8; ++e) {
            const __half2 v = *reinterpret_cast<const __half2*>(&hw[e]);
            big = __hmax2_nan(big, __habs2(v));
            f[e] = __half22float2(v);
          }
          if (p.interleaved) {
            // (x1, x2) (c, c) + (-x2, x1) (s, s)
#pragma unroll
            for (int e = 0; e < 8; ++e)
              f[e] = fma_f32x2(f[e], make_float2(cs[k][e], cs[k][e]),
                               mul_f32x2(make_float2(-f[e].y, f[e].x), make_float2(sn[k][e], sn[k][e])));
          } else {
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              const float2 u = f[e], v = f[e + 4];
              const float2 c = make_float2(cs[k][2 * e], cs[k][2 * e + 1]);
              const float2 d = make_float2(sn[k][2 * e], sn[k][2 * e + 1]);
              const float2 vd = mul_f32x2(v, d);
              f[e] = fma_f32x2(u, c, make_float2(-vd.x, -vd.y));
              f[e + 4] = fma_f32x2(v, c, mul_f32x2(u, d));
            }
          }
          if (__hbgt2(near, big)) {
#pragma unroll
            for (int e = 0; e < 8; ++e) split_near(f[e], hw[e], lw[e]);
          } else {
#pragma unroll
            for (int e = 0; e < 8; ++e) split_pair(f[e].x, f[e].y, hw[e], lw[e]);
          }
        }
        if (zero)
#pragma unroll
          for (int e = 0; e < 8; ++e) hw[e] = lw[e] = 0;
        __syncwarp();
        if (ok) {
          tmem_st4u(hi_tm + c0 * 4, hw);
          tmem_st4u(hi_tm + c1 * 4, hw + 4);
          tmem_st4u(lo_tm + c0 * 4, lw);
          tmem_st4u(lo_tm + c1 * 4, lw + 4);
        }
      }
      tmem_wait_st();
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(&turned[s]);
    }
  } else if (warp < kRpRotate + kRpStore) {
    // ------------------------------------------------------------------------- epilogue
    const int row = (warp & 3) * 32 + lane;
    const uint32_t trow = tmem + (static_cast<uint32_t>((warp & 3) * 32) << 16);
    const bool row_ok = n0 + row < n;
    int64_t slot = -1;
    if (!query && row_ok) {
      slot = p.slots[n0 + row];
      if (slot >= p.num_blocks * kBlockSize) {
        atomicOr(p.dev_err, RCP_DEVERR_BAD_SLOT);
        slot = -1;
      } else if (slot >= 0 && pos &&
                 static_cast<uint32_t>(pos[n0 + row]) >= static_cast<uint32_t>(p.num_pos)) {
        atomicOr(p.dev_err, RCP_DEVERR_BAD_POS);
        slot = -1;
      }
    }
    const int64_t blk = slot / kBlockSize, off = slot % kBlockSize;
    uint8_t* const pages = static_cast<uint8_t*>(p.k_pages);
    uint8_t* stage = sm + L::OUT_OFF + (warp - kRpRotate) * L::OUT_BYTES;
    // four warps take the even heads, four the odd ones
    for (int i = (warp - kRpRotate) >> 2; i < HG; i += 2) {
      const int s = i & 1, h = h0 + i;
      const int64_t run = (blk * S::H + h) * kBlockSize + off;   // the token's row of this head
      const bool ok = __all_sync(0xffffffffu, mbar_wait(&acc[s], (i >> 1) & 1, abort_flag, p.dev_err));
      tc_fence_after();
      if (!ok) break;
      const uint32_t tcol = trow + s * 64;
      auto load = [&](int c, float (&v)[16]) {
        tmem_ld16(tcol + c, v);
        tmem_wait_ld();
      };
      // 16 or 32 columns at a time: 832 threads have 72 registers each
      if (query && p.qhi == nullptr) {     // a decode's queries, fp32
        const size_t at = static_cast<size_t>(n0 + row) * S::H + h;
#pragma unroll
        for (int c = 0; c < RK; c += 16) {
          float v[16];
          load(c, v);
          uint4 w[4];
#pragma unroll
          for (int k = 0; k < 4; ++k)
            w[k] = make_uint4(__float_as_uint(v[4 * k] * p.qscale), __float_as_uint(v[4 * k + 1] * p.qscale),
                              __float_as_uint(v[4 * k + 2] * p.qscale),
                              __float_as_uint(v[4 * k + 3] * p.qscale));
          store_rows<4>(stage, lane, w, row_ok ? reinterpret_cast<uint8_t*>(p.qt + at * RK + c) : nullptr);
        }
      } else if (query) {                  // a prefill's, fp16 hi and lo, zero past r_k
        const size_t at = static_cast<size_t>(n0 + row) * S::H + h;
#pragma unroll
        for (int c0 = 0; c0 < 64; c0 += 32) {
          uint4 wh[4] = {}, wl[4] = {};
#pragma unroll
          for (int c = 0; c < 32; c += 16) {
            if (c0 + c >= RK) continue;
            float v[16];
            load(c0 + c, v);
            uint32_t hw[8], lw[8];
#pragma unroll
            for (int k = 0; k < 8; ++k)
              split_near(make_float2(v[2 * k] * p.qscale, v[2 * k + 1] * p.qscale), hw[k], lw[k]);
#pragma unroll
            for (int k = 0; k < 2; ++k) {
              wh[c / 8 + k] = make_uint4(hw[4 * k], hw[4 * k + 1], hw[4 * k + 2], hw[4 * k + 3]);
              wl[c / 8 + k] = make_uint4(lw[4 * k], lw[4 * k + 1], lw[4 * k + 2], lw[4 * k + 3]);
            }
          }
          const size_t to = at * 128 + c0 * 2;
          store_rows<4>(stage, lane, wh, row_ok ? static_cast<uint8_t*>(p.qhi) + to : nullptr);
          store_rows<4>(stage, lane, wl, row_ok ? static_cast<uint8_t*>(p.qlo) + to : nullptr);
        }
      } else if (p.page_format == RCP_PAGES_INT4) {
        using P = Int4Page<S>;
        float most = 0.f;
#pragma unroll 1
        for (int c = 0; c < RK; c += 16) {
          float v[16];
          load(c, v);
#pragma unroll
          for (int k = 0; k < 16; ++k) most = fmaxf(most, fabsf(v[k]));
        }
        const __half sh = int4_scale(most);
        const float sf = __half2float(sh), inv = __fdividef(1.f, sf);
        const int64_t r = h * kBlockSize + off;
        uint32_t* out = reinterpret_cast<uint32_t*>(pages + blk * P::KBYTES + r * RK / 2);
#pragma unroll 1
        for (int c = 0; c < RK; c += 16) {
          float v[16];
          __syncwarp();   // lanes without a slot have not stored
          load(c, v);
          uint32_t w[2] = {};
#pragma unroll
          for (int k = 0; k < 16; ++k) {
            const int code = sf > 0.f ? max(-7, min(7, rne_div(v[k], sf, inv))) : 0;
            w[k / 8] |= static_cast<uint32_t>(code & 0xF) << (4 * (k % 8));
          }
          if (slot >= 0) {
            out[c / 8] = w[0];
            out[c / 8 + 1] = w[1];
          }
        }
        if (slot >= 0) reinterpret_cast<__half*>(pages + blk * P::KBYTES + P::KCODES)[r] = sh;
        __syncwarp();
      } else if (p.page_format == RCP_PAGES_FP8_E4M3) {
        uint4 w[RK / 16];
#pragma unroll
        for (int c = 0; c < RK; c += 16) {
          float v[16];
          load(c, v);
          uint32_t b[4];
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            const float* x = &v[4 * k];
            b[k] = __nv_cvt_float2_to_fp8x2(make_float2(x[0], x[1]), __NV_SATFINITE, __NV_E4M3) |
                   static_cast<uint32_t>(
                       __nv_cvt_float2_to_fp8x2(make_float2(x[2], x[3]), __NV_SATFINITE, __NV_E4M3))
                       << 16;
          }
          w[c / 16] = make_uint4(b[0], b[1], b[2], b[3]);
        }
        store_rows<RK / 16>(stage, lane, w, slot >= 0 ? pages + run * RK : nullptr);
      } else {
        uint4 w[RK / 8];
#pragma unroll
        for (int c = 0; c < RK; c += 16) {
          float v[16];
          load(c, v);
          uint32_t b[8];
#pragma unroll
          for (int k = 0; k < 8; ++k) {
            const __half2 a = __floats2half2_rn(v[2 * k], v[2 * k + 1]);
            b[k] = *reinterpret_cast<const uint32_t*>(&a);
          }
          w[c / 8] = make_uint4(b[0], b[1], b[2], b[3]);
          w[c / 8 + 1] = make_uint4(b[4], b[5], b[6], b[7]);
        }
        store_rows<RK / 8>(stage, lane, w, slot >= 0 ? pages + run * RK * 2 : nullptr);
      }
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(&drained[s]);
    }
  } else if (warp == kRpRotate + kRpStore) {
    // --------------------------------------------------------------------------- copies
    if (lane == 0) {
      const CUtensorMap* xmap = query ? &q_map : &k_map;
      prefetch_tmap(xmap);
      prefetch_tmap(&u_map);
      int issued = 0;
      for (int i = 0; i < HG; ++i) {
        const int s = i % NS;
        if (i >= NS && !mbar_wait(&empty[s], ((i / NS) - 1) & 1, abort_flag, p.dev_err)) break;
        uint8_t* st = sm + s * L::STAGE;
        mbar_arrive_expect_tx(&full[s], L::STAGE);
        for (int kb = 0; kb < KB; ++kb) {
          tma_load_2d(st + kb * 128 * 128, xmap, (h0 + i) * D + kb * 64, n0, &full[s]);
          tma_load_2d(st + L::X_BYTES + kb * 64 * 128, &u_map, kb * 64, (h0 + i) * RK, &full[s]);
        }
        issued = i + 1;
      }
      for (int i = max(0, issued - NS); i < issued; ++i) mbar_wait_drain(&full[i % NS], (i / NS) & 1);
    }
  } else if (lane == 0) {
    // ----------------------------------------------------------------------------- MMAs
    constexpr uint32_t idesc = make_idesc_f16(128, RK, false, false);
    int done = 0;
    for (int i = 0; i < HG; ++i) {
      const int s = i & 1;
      if (i >= 2 && !mbar_wait(&drained[s], ((i >> 1) - 1) & 1, abort_flag, p.dev_err)) break;
      if (!mbar_wait(&turned[s], (i >> 1) & 1, abort_flag, p.dev_err)) break;
      tc_fence_after();
      const uint32_t u0 = smem_u32(sm + (i % NS) * L::STAGE + L::X_BYTES);
      const uint32_t hi_tm = tmem + L::A_TM + s * D;
#pragma unroll
      for (int k = 0; k < 4 * KB; ++k) {   // K = 16 steps: eight columns of the operand
        const uint64_t bd = make_sdesc(u0 + (k >> 2) * 64 * 128 + (k & 3) * 32, 16, 1024, kSwizzle128B);
        umma_f16_ta(tmem + s * 64, hi_tm + k * 8, bd, idesc, k > 0 ? 1u : 0u);
        if (pos) umma_f16_ta(tmem + s * 64, hi_tm + D / 2 + k * 8, bd, idesc, 1u);
      }
      umma_commit(&empty[i % NS]);
      umma_commit(&acc[s]);
      done = i + 1;
    }
    for (int i = max(0, done - 2); i < done; ++i) mbar_wait_drain(&acc[i & 1], (i >> 1) & 1);
  }
  __syncwarp();
  tc_fence_before();
  __syncthreads();
  if (warp == kRpRotate + kRpStore + 1) {
    tc_fence_after();
    tmem_dealloc(tmem, L::TMEM_COLS);
  }
  if ((behind_values || p.wait_at_exit) && blockIdx.x == 0) griddep_wait();
}

template <class S>
cudaError_t prepare_rotated_proj() {
  return cudaFuncSetAttribute(rotated_proj_kernel<S>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                              RpSmem<S>::ALLOC);
}

template <class S>
cudaError_t launch_rotated_proj(const CUtensorMap& u_k, const CUtensorMap& k_rows,
                                const CUtensorMap& q_rows, const AppendParams& p,
                                bool behind_values, cudaStream_t stream) {
  const int key_tiles = (p.T + 127) / 128, tiles = key_tiles + (p.nq + 127) / 128;
  return launch_pdl(rotated_proj_kernel<S>, dim3(tiles * p.proj_groups), dim3(kRpThreads),
                    RpSmem<S>::ALLOC, stream, true, u_k, k_rows, q_rows, p, key_tiles,
                    behind_values ? 1 : 0);
}

template cudaError_t prepare_rotated_proj<ShapeMain>();
template cudaError_t prepare_rotated_proj<ShapeTiny>();
template cudaError_t launch_rotated_proj<ShapeMain>(const CUtensorMap&, const CUtensorMap&,
                                                    const CUtensorMap&, const AppendParams&, bool,
                                                    cudaStream_t);
template cudaError_t launch_rotated_proj<ShapeTiny>(const CUtensorMap&, const CUtensorMap&,
                                                    const CUtensorMap&, const AppendParams&, bool,
                                                    cudaStream_t);

}  // namespace rcp
