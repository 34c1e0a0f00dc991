// Linear attention with one decay per head, one to eight tokens per call, on a
// [pool, H_v, D_k, D_v] state pool. With n of an item's L tokens committed,
//   o_t = scale (lambda^{t+1} S_0^T q_t + sum_{s <= t} lambda^{t-s} (q_t.k_s) v_s)
//   S_n = lambda^n S_0 + sum_{s < n} lambda^{n-1-s} k_s v_s^T
// so every state value is read once and written once, 4 bytes of traffic, and
// takes 2 L multiply-adds. A block owns up to 32 KB of one head's state: it
// arrives by TMA while the block prepares its tokens, is replaced in place in
// shared memory, and leaves by TMA. Four blocks an SM keep 128 KB in flight,
// and HBM bounds the call: 4.4 GB (512 items of 64 heads, 1 token, 64 x 512) in
// 670 to 731 us by the GPU, 6.0 to 6.5 TB/s; 290 MB (128 items of 32 heads, 8
// tokens, 128 x 128) in 52 us, 5.6 TB/s (46 us with the products left out).
//
// The multiply-adds run on mma.sync (m16n8k16, bf16 in, fp32 out), whose
// operands the 16 x 16 pieces of the tile are anyway after two ldmatrix, at
// a tenth of the instructions of an fp32 loop (which took 138 us where this
// takes 52, 128 items of 32 heads, 8 tokens, 128 x 128):
//   S_0^T q      both are bf16 as they are stored, so the products are exact;
//   sum k v^T    K = 16 holds the 8 weighted keys as bf16 hi and lo parts (16
//                significant bits) against the 8 values twice; the accumulator
//                starts from lambda^n S_0 in fp32;
//   q.k          exact products, fp32 sums.
// The tokens' own terms (8 x 8 scalars against v) are fp32 multiply-adds. The
// state is rounded to bf16 once, on its way back to the tile.
//
// Tokens that are not committed have weight 0 in the state and later tokens
// none in an output, and their values, which may be infinite, are masked there
// rather than multiplied by 0. A committed infinity may come out of the sum as a
// NaN: its own lo part is one, and the lo part 0 of a key times it is another.
#pragma once

#include <cuda.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include "gdr_linear.cuh"
#include "gdr_ptx.cuh"
#include "gdr_umma.cuh"

namespace gdr {

constexpr int kLdThreads = 128;  // 4 warps; of 128 columns, warp w takes strips w and w + 4
constexpr int kLdTileBytes = 32768;
constexpr int kLdPass = 128;     // columns worked on at a time

// n / d for 0 <= n < 2^31 by a product: q = (hi(n mul) + n) >> shift with
// shift = ceil(log2 d) and mul = floor(2^32 (2^shift - d) / d) + 1.
struct FastDiv {
  uint32_t mul, shift, d;
  __host__ static FastDiv by(uint32_t d) {
    uint32_t s = 0;
    while ((1ull << s) < d) ++s;
    return {static_cast<uint32_t>(((1ull << 32) * ((1ull << s) - d)) / d + 1), s, d};
  }
  __device__ __forceinline__ int div(int n) const {
    return static_cast<int>((__umulhi(static_cast<uint32_t>(n), mul) + static_cast<uint32_t>(n)) >>
                            shift);
  }
};

// Shared memory of a block of `cols` columns for T tokens: the tile, q and k
// [T][D_k + 8], the weighted keys [D_k][hi 8 | lo 8], v [T][cols + 8] (bf16; the
// row strides, and a swap of the keys' halves every four rows, put the 8 rows of a
// fragment into different banks), the 8 x 8 products of q and k, the powers of
// lambda, and S^T q of one pass [T][128] (fp32).
template <int DK>
struct LdShape {
  static constexpr int kMaxCols = kLdTileBytes / (2 * DK);  // 256 or 128
  static constexpr int kTokStride = DK + 8;
  int cols, T;
  __host__ __device__ LdShape(int cols_, int T_) : cols(cols_), T(T_) {}
  __host__ __device__ int val_stride() const { return cols + 8; }
  __host__ __device__ int q() const { return DK * cols * 2; }
  __host__ __device__ int k() const { return q() + T * kTokStride * 2; }
  __host__ __device__ int key() const { return k() + T * kTokStride * 2; }
  __host__ __device__ int val() const { return key() + DK * 32; }
  __host__ __device__ int a() const { return val() + T * val_stride() * 2; }
  __host__ __device__ int pow() const { return a() + 8 * 8 * 4; }
  __host__ __device__ int out() const { return pow() + 48; }
  __host__ __device__ int bar() const { return out() + T * kLdPass * 4; }
  __host__ __device__ int smem() const { return 1024 /* alignment slack */ + bar() + 16; }
};

struct LinearDecodeParams {
  LinearParams p;
  int part_cols;  // columns of a block, a multiple of 64 up to LdShape::kMaxCols
  FastDiv parts, heads, group;  // of D_v, H_v, and value heads of a query head
};

// D += A B, A 16 x 16 (row), B 16 x 8 (column), bf16 in, fp32 out.
__device__ __forceinline__ void mma_16816(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2,
                                          uint32_t a3, uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, "
      "{%8, %9}, {%0, %1, %2, %3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// A wait for copies of this CTA that are in flight, with the budget of the
// abandonable waits (gdr_ptx.cuh); nobody else can fail in between.
__device__ __forceinline__ bool mbar_wait_abandonable_alone(uint32_t bar, uint32_t parity) {
  const long long limit = abandonable_wait_limit();
  const long long t0 = clock64();
  while (!mbar_try_wait_suspend(bar, parity, kWaitSuspendNs))
    if (clock64() - t0 > limit) return false;
  return true;
}

// Blocks an SM: 5 where the registers decide (512 items of 64 heads, 64 x 512:
// 670 us against 679 for 4 on one GPU); at D_k = 128 shared memory leaves room for 4, and
// the registers of 4 are faster (8 tokens, 128 x 128: 52 us against 55).
template <int DK>
__global__ void __launch_bounds__(kLdThreads, DK == 128 ? 4 : 5)
    linear_decode_kernel(const __grid_constant__ CUtensorMap pool_map,
                         const LinearDecodeParams prm) {
  constexpr int KB = DK / 16;
  const LinearParams& p = prm.p;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int bh = prm.parts.div(static_cast<int>(blockIdx.x));
  const int col0 = (static_cast<int>(blockIdx.x) - bh * static_cast<int>(prm.parts.d)) *
                   prm.part_cols;
  const int b = prm.heads.div(bh), h = bh - b * p.H_v;
  const int cols = p.D_v - col0 < prm.part_cols ? p.D_v - col0 : prm.part_cols;
  const int T = p.T;

  extern __shared__ __align__(16) uint8_t smem_raw[];
  const uint32_t raw = smem_addr(smem_raw);
  uint8_t* smem = smem_raw + (((raw + 1023u) & ~1023u) - raw);
  const LdShape<DK> shape(prm.part_cols, T);
  constexpr int tok_stride = LdShape<DK>::kTokStride;
  const int v_stride = shape.val_stride();
  const uint32_t tile = smem_addr(smem);
  uint16_t* q_s = reinterpret_cast<uint16_t*>(smem + shape.q());
  uint16_t* k_s = reinterpret_cast<uint16_t*>(smem + shape.k());
  uint8_t* key_s = smem + shape.key();
  uint16_t* v_s = reinterpret_cast<uint16_t*>(smem + shape.val());
  float* a_s = reinterpret_cast<float*>(smem + shape.a());
  float* pw = reinterpret_cast<float*>(smem + shape.pow());  // lambda^0 .. lambda^8
  float* o_s = reinterpret_cast<float*>(smem + shape.out());
  const uint32_t bar = smem_addr(smem + shape.bar());

  // q, k and v are on their way before the item's slot is known: thread -> token
  // and 16-byte piece of its row
  constexpr int kPieces = DK / 8;
  uint4 q_r = make_uint4(0u, 0u, 0u, 0u), k_r = q_r, v_r[2] = {q_r, q_r};
  const int qk_at = tid / kPieces * tok_stride + tid % kPieces * 8;
  const bool has_qk = tid < T * kPieces;
  if (has_qk) {
    const size_t at = static_cast<size_t>(prm.group.div(bh)) * T * DK + tid * 8;
    q_r = *reinterpret_cast<const uint4*>(p.query + at);
    k_r = *reinterpret_cast<const uint4*>(p.key + at);
  }
  const int v_t = tid >> 4, v_c = (tid & 15) * 8;  // and columns v_c + 128
  if (v_t < T) {
    const uint16_t* value = p.value + (static_cast<size_t>(bh) * T + v_t) * p.D_v + col0 + v_c;
    if (v_c < cols) v_r[0] = *reinterpret_cast<const uint4*>(value);
    if (v_c + 128 < cols) v_r[1] = *reinterpret_cast<const uint4*>(value + 128);
  }
  const float log_decay = p.log_decay[h];
  int s, L, n;
  linear_item(p, b, s, L, n);
  uint16_t* out = p.out + static_cast<size_t>(bh) * T * p.D_v + col0;
  if (L == 0) {  // empty or skipped: +0.0, the slot untouched
    if (v_t < T)
      for (int c = v_c; c < cols; c += 128)
        *reinterpret_cast<uint4*>(out + static_cast<size_t>(v_t) * p.D_v + c) =
            make_uint4(0u, 0u, 0u, 0u);
    return;
  }
  const bool loads = !test_hold_tile(static_cast<int>(blockIdx.x));
  if (tid == 0) {
    mbar_init(bar, 1);
    fence_mbar_init();
    fence_async_smem();
    if (loads) {
      mbar_expect_tx(bar, cols / 64 * DK * 128);
      for (int x = 0; x < cols / 64; ++x)
        tma_load_3d(tile + x * DK * 128, &pool_map, col0 + 64 * x, 0, s * p.H_v + h, bar);
      mbar_arrive(bar);
    }
  }
  if (has_qk) {
    *reinterpret_cast<uint4*>(q_s + qk_at) = q_r;
    *reinterpret_cast<uint4*>(k_s + qk_at) = k_r;
  }
  if (v_t < T) {
    if (v_c < cols) *reinterpret_cast<uint4*>(v_s + v_t * v_stride + v_c) = v_r[0];
    if (v_c + 128 < cols) *reinterpret_cast<uint4*>(v_s + v_t * v_stride + v_c + 128) = v_r[1];
  }
  if (tid >= 96 && tid <= 96 + 8) pw[tid - 96] = decay_power(log_decay, tid - 96);
  __syncthreads();
  const int row = lane >> 2, pair = 2 * (lane & 3);  // a fragment's row and first column
  const int tok = row < T ? row : T - 1;  // rows behind T repeat the last: nothing reads them
  // q as the B operand of S^T q (and A of q k^T): token `row`, D_k 16 kb + pair ..
  const uint16_t* q_at = q_s + tok * tok_stride + pair;
  if (warp == 3) {  // a[t][u] = lambda^{t-u} q_t . k_u for u <= t
    const uint16_t* k_at = k_s + tok * tok_stride + pair;
    float d[2][4] = {};
#pragma unroll
    for (int kb = 0; kb < KB; ++kb)
      mma_16816(d[kb & 1], *reinterpret_cast<const uint32_t*>(q_at + 16 * kb), 0u,
                *reinterpret_cast<const uint32_t*>(q_at + 16 * kb + 8), 0u,
                *reinterpret_cast<const uint32_t*>(k_at + 16 * kb),
                *reinterpret_cast<const uint32_t*>(k_at + 16 * kb + 8));
#pragma unroll
    for (int e = 0; e < 2; ++e)
      if (pair + e <= row) a_s[row * 8 + pair + e] = (d[0][e] + d[1][e]) * pw[row - pair - e];
  }
  // the committed keys times lambda^{n-1-t}, as hi and lo: a thread a row
  if (tid < DK) {
    uint32_t hi[4] = {0u, 0u, 0u, 0u}, lo[4] = {0u, 0u, 0u, 0u};
#pragma unroll
    for (int c = 0; c < 4; ++c) {
      if (2 * c < n) {
        const float w0 = bf16_bits_to_f32(k_s[2 * c * tok_stride + tid]) * pw[n - 1 - 2 * c];
        const float w1 = 2 * c + 1 < n ? bf16_bits_to_f32(k_s[(2 * c + 1) * tok_stride + tid]) *
                                             pw[n - 2 - 2 * c]
                                       : 0.0f;
        hi[c] = pack_bf16x2(w0, w1);
        lo[c] = pack_bf16x2(w0 - bf16_lo(hi[c]), w1 - bf16_hi(hi[c]));
      }
    }
    uint4* dst = reinterpret_cast<uint4*>(key_s + tid * 32);
    dst[(tid >> 2) & 1] = make_uint4(hi[0], hi[1], hi[2], hi[3]);
    dst[((tid >> 2) & 1) ^ 1] = make_uint4(lo[0], lo[1], lo[2], lo[3]);
  }
  __syncthreads();
  const bool landed = mbar_wait_abandonable_alone(bar, 0);
  if (!__syncthreads_and(landed)) {
    if (tid == 0) {
      flag_error(kErrConsumerWait);
      if (loads && !mbar_wait_bounded(bar, 0)) flag_error(kErrDrainWait);
    }
    return;
  }

  // masks of the committed ones of tokens pair and pair + 1
  const uint32_t committed = (pair < n ? 0xffffu : 0u) | (pair + 1 < n ? 0xffff0000u : 0u);
  const float lambda_n = pw[n];
  const unsigned long long ln2 = pk(lambda_n, lambda_n);
  const int m_row = (lane & 7) + (lane & 8);  // ldmatrix: row of the 16 x 16 piece
  const int m_chunk = lane >> 4;              // and its 8-column half
  const uint32_t key_at = smem_addr(key_s) + m_row * 32 + ((m_chunk ^ ((m_row >> 2) & 1)) << 4);
  const int v_row = (lane & 7) < T ? lane & 7 : T - 1;
  // four columns of a token a thread, for the outputs of a pass
  const int sh = T > 4 ? 4 : (T > 2 ? 5 : (T > 1 ? 6 : 7));
  const int t = tid >> sh;
  // The fragments of 16 rows: the state as stored and transposed, keys, q.
  struct Rows {
    uint32_t s[2][4], t[2][4], k[4], q[2];
  };
  for (int c0 = 0; c0 < cols; c0 += kLdPass) {
    const int strips = cols - c0 > 64 ? 2 : 1;
    // this lane's address of the strips' first pieces; a piece further down is 16 rows on
    uint32_t at[2], vf[2][2];
    float o[2][4];
#pragma unroll
    for (int j = 0; j < 2; ++j) {
      at[j] = tile + ((c0 >> 6) + j) * DK * 128 + m_row * 128 +
              (((2 * warp + m_chunk) ^ (m_row & 7)) << 4);
      vf[j][0] = vf[j][1] = 0u;
      if (j < strips) {  // the committed values as B operands, two 8-column tiles a strip
        ldmatrix_x2_trans(
            smem_addr(v_s + v_row * v_stride + c0 + 64 * j + 16 * warp + (lane & 8)), vf[j]);
        vf[j][0] &= committed;
        vf[j][1] &= committed;
      }
#pragma unroll
      for (int e = 0; e < 4; ++e) o[j][e] = 0.0f;
    }
    const auto fetch = [&](int kb, Rows& f) {
      ldmatrix_x4(key_at + kb * 512, f.k);
      f.q[0] = *reinterpret_cast<const uint32_t*>(q_at + 16 * kb);
      f.q[1] = *reinterpret_cast<const uint32_t*>(q_at + 16 * kb + 8);
#pragma unroll
      for (int j = 0; j < 2; ++j)
        if (j < strips) {
          ldmatrix_x4(at[j] + kb * 2048, f.s[j]);
          ldmatrix_x4_trans(at[j] + kb * 2048, f.t[j]);
        }
    };
    const auto work = [&](int kb, const Rows& f) {
      // both strips' products first, then their roundings: the products of one
      // run under those of the other
      float d[2][2][4];
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        if (j < strips) {
          mma_16816(o[j], f.t[j][0], f.t[j][2], f.t[j][1], f.t[j][3], f.q[0], f.q[1]);
#pragma unroll
          for (int c = 0; c < 2; ++c) {
#pragma unroll
            for (int e = 0; e < 2; ++e) {
              const uint32_t x = f.s[j][2 * c + e];
              const float2 y = upk(mul2(ln2, pk(bf16_lo(x), bf16_hi(x))));
              d[j][c][2 * e] = y.x;
              d[j][c][2 * e + 1] = y.y;
            }
            mma_16816(d[j][c], f.k[0], f.k[1], f.k[2], f.k[3], vf[j][c], vf[j][c]);
          }
        }
      }
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        if (j < strips && n > 0) {
          const uint32_t y[4] = {pack_bf16x2(d[j][0][0], d[j][0][1]),
                                 pack_bf16x2(d[j][0][2], d[j][0][3]),
                                 pack_bf16x2(d[j][1][0], d[j][1][1]),
                                 pack_bf16x2(d[j][1][2], d[j][1][3])};
          stmatrix_x4(at[j] + kb * 2048, y);
        }
      }
    };
    // the next 16 rows are fetched before these are worked on
    Rows even, odd;
    fetch(0, even);
#pragma unroll 1
    for (int kb = 0; kb < KB; kb += 2) {
      fetch(kb + 1, odd);
      work(kb, even);
      if (kb + 2 < KB) fetch(kb + 2, even);
      work(kb + 1, odd);
    }
    // o[j]: columns row and row + 8 of the strip, tokens pair and pair + 1
#pragma unroll
    for (int j = 0; j < 2; ++j)
      if (j < strips) {
#pragma unroll
        for (int e = 0; e < 4; ++e)
          if (pair + (e & 1) < T)
            o_s[(pair + (e & 1)) * kLdPass + 64 * j + 16 * warp + row + 8 * (e >> 1)] = o[j][e];
      }
    fence_async_smem();
    __syncthreads();
    if (tid == 0 && n > 0) {  // these columns of the state leave
      for (int x = c0 >> 6; x < (c0 >> 6) + strips; ++x)
        tma_store_3d(&pool_map, col0 + 64 * x, 0, s * p.H_v + h, tile + x * DK * 128);
      bulk_commit_group();
    }
    // the tokens' own terms, and the outputs
    if (t < T) {
      const int pass = 64 * strips;
      for (int c = (tid & ((1 << sh) - 1)) * 4; c < pass; c += 4 << sh) {
        uint2 y = make_uint2(0u, 0u);  // padding: +0.0
        if (t < L) {
          const float4 f = *reinterpret_cast<const float4*>(o_s + t * kLdPass + c);
          const float decay = pw[t + 1];
          float x[4] = {f.x * decay, f.y * decay, f.z * decay, f.w * decay};
          for (int u = 0; u <= t; ++u) {
            const float a = a_s[t * 8 + u];
            const uint2 w = *reinterpret_cast<const uint2*>(v_s + u * v_stride + c0 + c);
            x[0] = fmaf(a, bf16_lo(w.x), x[0]);
            x[1] = fmaf(a, bf16_hi(w.x), x[1]);
            x[2] = fmaf(a, bf16_lo(w.y), x[2]);
            x[3] = fmaf(a, bf16_hi(w.y), x[3]);
          }
          y = make_uint2(pack_bf16x2(x[0] * p.scale, x[1] * p.scale),
                         pack_bf16x2(x[2] * p.scale, x[3] * p.scale));
        }
        *reinterpret_cast<uint2*>(out + static_cast<size_t>(t) * p.D_v + c0 + c) = y;
      }
    }
    if (c0 + kLdPass < cols) __syncthreads();  // o_s is written again
  }
  if (tid == 0) bulk_wait_read_all();
}

}  // namespace gdr
