// Linear attention with one decay per head over prompts of any length, in the
// chunk form on the tensor cores. For a chunk of C = 128 tokens that starts
// from state S (lambda the head's decay, i and j positions in the chunk):
//   P_ij = lambda^{i-j} (q_i . k_j) for j <= i, else 0
//   O_i  = scale (sum_j P_ij v_j + lambda^{i+1} S^T q_i)
//   S   <- lambda^C S + sum_j lambda^{C-1-j} k_j v_j^T
// so 4 products of 128 x 128 x 128 a chunk, head and 128 columns of v stand
// for 128 dependent steps. No power of lambda is ever divided by: each one
// has an exponent >= 0, so nothing overflows for lambda <= 1 and a decay of
// zero is exact.
//
// A CTA takes one (item, value head, 128 columns of D_v) and walks its chunks.
// TMEM (512 columns, fp32): P | S^T q | P V | the state, transposed (lane = a
// column j of S). Roles, one warp or one group of four warps each:
//   load     TMA of the chunk's q, k, v into a ring of stages;
//   mma      the four products: P = q k^T; S^T q; S += (V^T)(weighted k);
//            P V with P read from TMEM;
//   P        P out of TMEM, times lambda^{i-j}, masked, back as bf16 over
//            itself;
//   out      (S^T q) lambda^{i+1} + P V, scaled, to bf16 in the chunk's v stage
//            (both products have read v by then), TMA store;
//   state    k in place times lambda^{C-1-j}; then S out of TMEM to bf16 in
//            shared memory for the next chunk's S^T q, and back scaled by
//            lambda^C for the next chunk's sum.
// The mma warp issues the next chunk's q k^T right behind this chunk's P V, so
// the tensor pipe waits only where the chain through the state is longer.
//
// Roundings to bf16, next to the fp32 sums: P and the weighted k, since the
// other operand of their products is bf16 and one MMA takes one type; and the
// copy of S that S^T q reads. Each is at most 2^-8 of its term, with a
// random sign, about what the bf16 output's own rounding adds. The state
// itself stays fp32 from the first chunk to the last.
//
// Rows behind an item's last token: k is weighted 0 and v zeroed by a write
// (not a product: padding may hold NaN), q only reaches rows that are written
// as zeros. P's masked entries are written as 0, not multiplied by 0.
//
// Waits follow the failure protocol of gdr_ptx.cuh: each is bounded, a failed
// one ends its role (by vote where a group has a barrier), nothing is signalled
// after a failure, and copies and MMAs in flight are waited for before the
// tensor memory is freed.
#pragma once

#include <cuda.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include "gdr_linear.cuh"
#include "gdr_ptx.cuh"
#include "gdr_umma.cuh"

namespace gdr {

constexpr int kLpChunk = 128;              // tokens of a chunk
constexpr int kLpCols = 128;               // columns of D_v of a CTA
constexpr int kLpThreads = 512;
constexpr int kLpBox = kLpChunk * 128;     // bytes of 128 rows x 64 bf16
constexpr int kLpTmemCols = 512;
constexpr int kLpTmemP = 0, kLpTmemInter = 128, kLpTmemIntra = 256, kLpTmemState = 384;
constexpr int kLpBars = 8;                 // besides three per stage

template <int DK>
struct LpShape {
  static constexpr int kBoxes = DK / 64;                  // 64-column boxes of q and of k
  static constexpr int kStages = DK == 128 ? 2 : 3;
  static constexpr int kStageBytes = (2 * kBoxes + 2) * kLpBox;  // q, k, v
  static constexpr int kStateOff = kStages * kStageBytes;        // bf16 S^T, [128 j][DK]
  static constexpr int kBarOff = kStateOff + kBoxes * kLpBox;
  static constexpr int kPowOff = kBarOff + 8 * (3 * kStages + kLpBars) + 16;
  static constexpr int kSmem = 1024 + kPowOff + 4 * (kLpChunk + 1);
};

struct LinearPrefillParams {
  LinearParams p;
  int slices;      // ceil(D_v / 128)
};

// Byte offset of 16-byte chunk c (8 bf16) of row r in a [128 rows][64 columns]
// box with the 128-byte swizzle.
__device__ __forceinline__ int lp_swz(int r, int c) { return r * 128 + ((c ^ (r & 7)) << 4); }

template <int DK>
__global__ void __launch_bounds__(kLpThreads, 1)
    linear_prefill_kernel(const __grid_constant__ CUtensorMap q_map,
                          const __grid_constant__ CUtensorMap k_map,
                          const __grid_constant__ CUtensorMap v_map,
                          const __grid_constant__ CUtensorMap o_map,
                          const LinearPrefillParams prm) {
  using Shape = LpShape<DK>;
  constexpr int kBoxes = Shape::kBoxes, kStages = Shape::kStages;
  const LinearParams& p = prm.p;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int slice = blockIdx.x % prm.slices;
  const int bh = blockIdx.x / prm.slices;
  const int h = bh % p.H_v, b = bh / p.H_v;
  const int col0 = slice * kLpCols;
  const int cols = p.D_v - col0 < kLpCols ? p.D_v - col0 : kLpCols;  // 64 or 128
  int s, L, n;
  linear_item(p, b, s, L, n);
  uint16_t* out = p.out + static_cast<size_t>(bh) * p.T * p.D_v + col0;
  const int n_chunks = (L + kLpChunk - 1) / kLpChunk;
  if (L == 0) {  // empty or skipped: +0.0, the slot untouched
    const int per_row = cols / 8;
    for (int64_t e = tid; e < static_cast<int64_t>(p.T) * per_row; e += kLpThreads)
      *reinterpret_cast<uint4*>(out + (e / per_row) * p.D_v + (e % per_row) * 8) =
          make_uint4(0u, 0u, 0u, 0u);
    return;
  }

  extern __shared__ __align__(16) uint8_t smem_raw[];
  const uint32_t raw = smem_addr(smem_raw);
  uint8_t* smem = smem_raw + (((raw + 1023u) & ~1023u) - raw);
  uint64_t* bars = reinterpret_cast<uint64_t*>(smem + Shape::kBarOff);
  float* pw = reinterpret_cast<float*>(smem + Shape::kPowOff);  // lambda^0 .. lambda^128
  const uint32_t bar0 = smem_addr(bars);
  const uint32_t full = bar0;                      // + 8 st: q, k, v landed
  const uint32_t qk_free = bar0 + 8 * kStages;     // + 8 st: q and k read for the last time
  const uint32_t v_free = bar0 + 16 * kStages;     // + 8 st: the output has left the v stage
  const uint32_t bar1 = bar0 + 24 * kStages;
  const uint32_t p_raw = bar1, p_ready = bar1 + 8, k_ready = bar1 + 16, s_ready = bar1 + 24,
                 s_raw = bar1 + 32, o_raw = bar1 + 40, o_free = bar1 + 48, drained = bar1 + 56;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(bars + 3 * kStages + kLpBars);
  volatile int* abort_word = reinterpret_cast<volatile int*>(tmem_slot + 1);

  const float log_decay = p.log_decay[h];
  if (tid == 0) {
    for (int st = 0; st < kStages; ++st) {
      mbar_init(full + 8 * st, 1);
      mbar_init(qk_free + 8 * st, 1);
      mbar_init(v_free + 8 * st, 1);
    }
    mbar_init(p_raw, 1);
    mbar_init(p_ready, 128);
    mbar_init(k_ready, 128);
    mbar_init(s_ready, 128);
    mbar_init(s_raw, 1);
    mbar_init(o_raw, 1);
    mbar_init(o_free, 128);
    mbar_init(drained, 1);
    *abort_word = 0;
    fence_mbar_init();
  }
  if (tid >= 128 && tid <= 128 + kLpChunk) pw[tid - 128] = decay_power(log_decay, tid - 128);
  __syncwarp();
  if (warp == 0) {
    tmem_alloc(smem_addr(tmem_slot), kLpTmemCols);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;

  if (warp == 0) {
    // ------------------------------------------------------------ load
    if (lane == 0 && !test_hold_tile(static_cast<int>(blockIdx.x))) {
      const int zq = b * p.H_qk + h / p.group;
      const uint32_t bytes = (2 * kBoxes + cols / 64) * kLpBox;
      int issued = 0;
      for (int i = 0; i < n_chunks; ++i) {
        const int st = i % kStages;
        const uint32_t free_phase = ((i / kStages) & 1) ^ 1;
        if (!mbar_wait_abandonable(qk_free + 8 * st, free_phase, abort_word, kErrProducerWait) ||
            !mbar_wait_abandonable(v_free + 8 * st, free_phase, abort_word, kErrProducerWait))
          break;
        const uint32_t dst = smem_addr(smem + st * Shape::kStageBytes);
        mbar_expect_tx(full + 8 * st, bytes);
#pragma unroll
        for (int x = 0; x < kBoxes; ++x) {
          tma_load_3d(dst + x * kLpBox, &q_map, 64 * x, i * kLpChunk, zq, full + 8 * st);
          tma_load_3d(dst + (kBoxes + x) * kLpBox, &k_map, 64 * x, i * kLpChunk, zq,
                      full + 8 * st);
        }
        for (int x = 0; x < cols / 64; ++x)
          tma_load_3d(dst + (2 * kBoxes + x) * kLpBox, &v_map, col0 + 64 * x, i * kLpChunk, bh,
                      full + 8 * st);
        mbar_arrive(full + 8 * st);
        ++issued;
      }
      for (int i = issued > kStages ? issued - kStages : 0; i < issued; ++i)
        if (!mbar_wait_bounded(full + 8 * (i % kStages), (i / kStages) & 1)) {
          flag_error(kErrDrainWait);
          break;
        }
    }
  } else if (warp == 1) {
    // ------------------------------------------------------------ mma
    if (lane == 0) {
      constexpr uint32_t id_qk = umma_idesc_bf16<128, 128, false, false>();
      constexpr uint32_t id_pv = umma_idesc_bf16<128, 128, false, true>();
      constexpr uint32_t id_kv = umma_idesc_bf16<128, DK, true, true>();
      const uint64_t s_desc =
          umma_desc(smem_addr(smem + Shape::kStateOff), 16, 1024, kUmmaSwizzle128);
      auto wait = [&](uint32_t bar, uint32_t phase) {
        const bool ok = mbar_wait_abandonable(bar, phase, abort_word, kErrConsumerWait);
        tc_fence_after();
        return ok;
      };
      for (int i = 0; i < n_chunks; ++i) {
        const int st = i % kStages;
        const uint32_t ph = i & 1;
        const uint32_t q_s = smem_addr(smem + st * Shape::kStageBytes);
        const uint32_t k_s = q_s + kBoxes * kLpBox, v_s = k_s + kBoxes * kLpBox;
        const uint64_t q_k = umma_desc(q_s, 16, 1024, kUmmaSwizzle128);
        const uint64_t k_k = umma_desc(k_s, 16, 1024, kUmmaSwizzle128);
        const uint64_t k_mn = umma_desc(k_s, kLpBox, 1024, kUmmaSwizzle128);
        const uint64_t v_mn = umma_desc(v_s, kLpBox, 1024, kUmmaSwizzle128);
        if (!wait(full + 8 * st, (i / kStages) & 1)) break;
#pragma unroll
        for (int ks = 0; ks < DK / 16; ++ks) {
          const uint32_t off = (ks >> 2) * kLpBox + (ks & 3) * 32;
          umma_bf16(tmem + kLpTmemP, umma_desc_advance(q_k, off), umma_desc_advance(k_k, off),
                    id_qk, ks > 0);
        }
        umma_commit(p_raw);
        if (!wait(s_ready, ph)) break;
        if (i > 0 && !wait(o_free, ph ^ 1)) break;
#pragma unroll
        for (int ks = 0; ks < DK / 16; ++ks) {
          const uint32_t off = (ks >> 2) * kLpBox + (ks & 3) * 32;
          umma_bf16(tmem + kLpTmemInter, umma_desc_advance(q_k, off),
                    umma_desc_advance(s_desc, off), id_qk, ks > 0);
        }
        if (!wait(k_ready, ph)) break;
#pragma unroll
        for (int ks = 0; ks < kLpChunk / 16; ++ks)
          umma_bf16(tmem + kLpTmemState, umma_desc_advance(v_mn, ks * 2048),
                    umma_desc_advance(k_mn, ks * 2048), id_kv, true);
        umma_commit(s_raw);
        if (!wait(p_ready, ph)) break;
#pragma unroll
        for (int ks = 0; ks < kLpChunk / 16; ++ks)
          umma_bf16_ts(tmem + kLpTmemIntra, tmem + kLpTmemP + 8 * ks,
                       umma_desc_advance(v_mn, ks * 2048), id_pv, ks > 0);
        umma_commit(o_raw);
        umma_commit(qk_free + 8 * st);
      }
      umma_commit(drained);
      if (!mbar_wait_bounded(drained, 0)) flag_error(kErrDrainWait);
    }
  } else if (warp < 4) {
    // ------------------------------------------------------------ padding
    // tokens behind the last chunk: +0.0
    const int per_row = cols / 8;
    const int64_t end = static_cast<int64_t>(p.T) * per_row;
    for (int64_t e = static_cast<int64_t>(n_chunks) * kLpChunk * per_row + (tid - 64); e < end;
         e += 64)
      *reinterpret_cast<uint4*>(out + (e / per_row) * p.D_v + (e % per_row) * 8) =
          make_uint4(0u, 0u, 0u, 0u);
  } else if (warp < 8) {
    // ------------------------------------------------------------ P
    const int wq = warp & 3, t = tid & 127;
    const uint32_t base = tmem + kLpTmemP + (static_cast<uint32_t>(32 * wq) << 16);
    for (int i = 0; i < n_chunks; ++i) {
      const bool ok = mbar_wait_abandonable(p_raw, i & 1, abort_word, kErrConsumerWait);
      if (!__all_sync(0xffffffffu, ok)) break;
      tc_fence_after();
#pragma unroll 1
      for (int j = 0; j < 4; ++j) {
        uint32_t y[16];
        if (j <= wq) {  // columns 32 j .. of rows 32 wq ..: some are unmasked
          uint32_t x[32];
          tmem_ld32(base + 32 * j, x);
          tmem_wait_ld();
          const float* pt = pw + (t - 32 * j);
#pragma unroll
          for (int e = 0; e < 16; ++e) {
            const int c = 32 * j + 2 * e;
            const float a = c <= t ? __uint_as_float(x[2 * e]) * pt[-2 * e] : 0.0f;
            const float d = c + 1 <= t ? __uint_as_float(x[2 * e + 1]) * pt[-2 * e - 1] : 0.0f;
            y[e] = pack_bf16x2(a, d);
          }
        } else {
#pragma unroll
          for (int e = 0; e < 16; ++e) y[e] = 0u;
        }
        tmem_st16(base + 16 * j, y);
      }
      tmem_wait_st();
      tc_fence_before();
      mbar_arrive(p_ready);
    }
  } else if (warp < 12) {
    // ------------------------------------------------------------ out
    const int wq = warp & 3, t = tid & 127;
    const uint32_t lanes = tmem + (static_cast<uint32_t>(32 * wq) << 16);
    const float inter = pw[t + 1] * p.scale;
    const bool elected = t == 0;
    for (int i = 0; i < n_chunks; ++i) {
      const int st = i % kStages;
      const int Lc = L - i * kLpChunk;
      uint8_t* o_s = smem + st * Shape::kStageBytes + 2 * kBoxes * kLpBox;
      const bool ok =
          __all_sync(0xffffffffu, mbar_wait_abandonable(o_raw, i & 1, abort_word,
                                                        kErrConsumerWait));
      if (ok) {
        tc_fence_after();
#pragma unroll 1
        for (int j = 0; j < 4; ++j) {
          uint32_t x[32], z[32];
          tmem_ld32(lanes + kLpTmemInter + 32 * j, x);
          tmem_ld32(lanes + kLpTmemIntra + 32 * j, z);
          tmem_wait_ld();
#pragma unroll
          for (int c = 0; c < 4; ++c) {
            uint32_t y[4];
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              const int k = 8 * c + 2 * e;
              y[e] = t < Lc ? pack_bf16x2(fmaf(__uint_as_float(x[k]), inter,
                                               __uint_as_float(z[k]) * p.scale),
                                          fmaf(__uint_as_float(x[k + 1]), inter,
                                               __uint_as_float(z[k + 1]) * p.scale))
                            : 0u;
            }
            *reinterpret_cast<uint4*>(o_s + (j >> 1) * kLpBox + lp_swz(t, 4 * (j & 1) + c)) =
                make_uint4(y[0], y[1], y[2], y[3]);
          }
        }
        tc_fence_before();
        mbar_arrive(o_free);
      }
      fence_async_smem();
      if (!named_barrier_and(1, 128, ok)) break;
      if (elected) {
        for (int x = 0; x < cols / 64; ++x)
          tma_store_3d(&o_map, col0 + 64 * x, i * kLpChunk, bh, smem_addr(o_s + x * kLpBox));
        bulk_commit_group();
        bulk_wait_read_all();
        mbar_arrive(v_free + 8 * st);
      }
    }
    if (elected) bulk_wait_all();
  } else {
    // ------------------------------------------------------------ state
    const int wq = warp & 3, r = tid & 127;  // r: column j of S, row of k and v
    const uint32_t lanes = tmem + kLpTmemState + (static_cast<uint32_t>(32 * wq) << 16);
    uint8_t* s_s = smem + Shape::kStateOff;
    const bool live = r < cols;
    uint16_t* slot =
        p.state_pool + (static_cast<size_t>(s) * p.H_v + h) * DK * p.D_v + col0 + r;
    // the slot: bf16 as it is for the first S^T q, scaled into TMEM for the first sum
    {
      const float decay = pw[L < kLpChunk ? L : kLpChunk];
#pragma unroll 1
      for (int j = 0; j < DK / 32; ++j) {
        uint32_t x[32];
#pragma unroll
        for (int e = 0; e < 32; ++e)
          x[e] = live ? slot[static_cast<size_t>(32 * j + e) * p.D_v] : 0u;
#pragma unroll
        for (int c = 0; c < 4; ++c)
          *reinterpret_cast<uint4*>(s_s + (j >> 1) * kLpBox + lp_swz(r, 4 * (j & 1) + c)) =
              make_uint4(x[8 * c] | (x[8 * c + 1] << 16), x[8 * c + 2] | (x[8 * c + 3] << 16),
                         x[8 * c + 4] | (x[8 * c + 5] << 16),
                         x[8 * c + 6] | (x[8 * c + 7] << 16));
#pragma unroll
        for (int e = 0; e < 32; ++e) x[e] = __float_as_uint(__uint_as_float(x[e] << 16) * decay);
        tmem_st32(lanes + 32 * j, x);
      }
      tmem_wait_st();
      fence_async_smem();
      tc_fence_before();
      mbar_arrive(s_ready);
    }
    for (int i = 0; i < n_chunks; ++i) {
      const int st = i % kStages;
      const int left = L - i * kLpChunk;
      const int Lc = left < kLpChunk ? left : kLpChunk;
      uint8_t* k_s = smem + st * Shape::kStageBytes + kBoxes * kLpBox;
      uint8_t* v_s = k_s + kBoxes * kLpBox;
      bool ok = mbar_wait_abandonable(full + 8 * st, (i / kStages) & 1, abort_word,
                                      kErrConsumerWait) &&
                mbar_wait_abandonable(p_raw, i & 1, abort_word, kErrConsumerWait);
      if (!__all_sync(0xffffffffu, ok)) break;
      // row r of k times lambda^{Lc-1-r}. Lanes start at different 16-byte
      // pieces of their rows, so that 8 lanes of a row group hit 8 bank groups.
      const float weight = r < Lc ? pw[Lc - 1 - r] : 0.0f;
#pragma unroll
      for (int x = 0; x < kBoxes; ++x)
#pragma unroll
        for (int c = 0; c < 8; ++c) {
          uint4* at = reinterpret_cast<uint4*>(k_s + x * kLpBox + lp_swz(r, c));
          uint4 w = *at;
          uint32_t y[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
          for (int e = 0; e < 4; ++e)
            y[e] = r < Lc ? pack_bf16x2(bf16_lo(y[e]) * weight, bf16_hi(y[e]) * weight) : 0u;
          *at = make_uint4(y[0], y[1], y[2], y[3]);
        }
      if (r >= Lc) {
#pragma unroll
        for (int c = 0; c < 16; ++c)
          *reinterpret_cast<uint4*>(v_s + (c >> 3) * kLpBox + lp_swz(r, c & 7)) =
              make_uint4(0u, 0u, 0u, 0u);
      }
      fence_async_smem();
      mbar_arrive(k_ready);

      ok = mbar_wait_abandonable(s_raw, i & 1, abort_word, kErrConsumerWait);
      if (!__all_sync(0xffffffffu, ok)) break;
      tc_fence_after();
      const bool last = i + 1 == n_chunks;
      const float decay = pw[left - Lc < kLpChunk ? left - Lc : kLpChunk];
#pragma unroll 1
      for (int j = 0; j < DK / 32; ++j) {
        uint32_t x[32];
        tmem_ld32(lanes + 32 * j, x);
        tmem_wait_ld();
        if (last) {
          if (live) {
#pragma unroll
            for (int e = 0; e < 32; ++e)
              slot[static_cast<size_t>(32 * j + e) * p.D_v] =
                  f32_to_bf16_bits(__uint_as_float(x[e]));
          }
          continue;
        }
#pragma unroll
        for (int c = 0; c < 4; ++c) {
          uint32_t y[4];
#pragma unroll
          for (int e = 0; e < 4; ++e)
            y[e] = pack_bf16x2(__uint_as_float(x[8 * c + 2 * e]),
                               __uint_as_float(x[8 * c + 2 * e + 1]));
          *reinterpret_cast<uint4*>(s_s + (j >> 1) * kLpBox + lp_swz(r, 4 * (j & 1) + c)) =
              make_uint4(y[0], y[1], y[2], y[3]);
        }
#pragma unroll
        for (int e = 0; e < 32; ++e) x[e] = __float_as_uint(__uint_as_float(x[e]) * decay);
        tmem_st32(lanes + 32 * j, x);
      }
      if (!last) {
        tmem_wait_st();
        fence_async_smem();
        tc_fence_before();
        mbar_arrive(s_ready);
      }
    }
  }

  // every warp arrives here: free the tensor memory once no thread can touch it
  __syncwarp();
  tc_fence_before();
  __syncthreads();
  if (warp == 0) {
    tc_fence_after();
    tmem_dealloc(tmem, kLpTmemCols);
  }
}

}  // namespace gdr
