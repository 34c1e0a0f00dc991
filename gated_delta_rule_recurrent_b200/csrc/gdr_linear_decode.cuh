// Linear attention with one decay per head, one to eight tokens per call, on a
// [pool, H_v, D_k, D_v] state pool.
//
// Both kernels read each state value once and write it once; at 4 bytes of
// traffic a value the time is HBM's as long as enough loads are in flight.
//
// One token: s' = lambda s + k_i v_j and o_j = scale sum_i q_i s'_ij. A warp
// owns 64 columns of a head: 8 lanes of 8 columns (16 bytes) by 4 row groups,
// so the sum over rows is two shuffles a column at the end, and nothing is
// staged in shared memory. For small calls RS warps share the rows of a tile
// (their sums meet in shared memory), which shortens each warp's chain of
// loads.
//
// Several tokens, in the chunk form: with n of L tokens committed,
//   o_t = scale (lambda^{t+1} S_0^T q_t + sum_{s <= t} lambda^{t-s} (q_t.k_s) v_s)
//   S_n = lambda^n S_0 + sum_{s < n} lambda^{n-1-s} k_s v_s^T
// so a state value takes 2 L multiply-adds and no chain over the tokens. The
// tokens go in pairs through the packed fp32 instructions (two multiply-adds
// an issue slot): at L = 8 a value costs about 13 issue slots where the HBM
// time of its 4 bytes leaves 22.
//
// Everything is fp32; the state is rounded to bf16 once, on the store.
#pragma once

#include <cuda_runtime.h>
#include <stdint.h>

#include "gdr_linear.cuh"
#include "gdr_ptx.cuh"

namespace gdr {

constexpr int kLinOneThreads = 128;  // 4 warps

// N consecutive bf16 (N = 4, 8 or a multiple of 8) as fp32; aligned to 2 N
// bytes (16 at most).
template <int N>
__device__ __forceinline__ void load_bf16(const uint16_t* src, float (&dst)[N]) {
  if constexpr (N == 4) {
    const uint2 w = *reinterpret_cast<const uint2*>(src);
    dst[0] = bf16_lo(w.x);
    dst[1] = bf16_hi(w.x);
    dst[2] = bf16_lo(w.y);
    dst[3] = bf16_hi(w.y);
  } else {
#pragma unroll
    for (int c = 0; c < N / 8; ++c) {
      const uint4 w = reinterpret_cast<const uint4*>(src)[c];
      const uint32_t x[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        dst[8 * c + 2 * e] = bf16_lo(x[e]);
        dst[8 * c + 2 * e + 1] = bf16_hi(x[e]);
      }
    }
  }
}

// One token. RS warps (1 or 4) of a block share a 64-column tile.
template <int DK, int RS>
__global__ void __launch_bounds__(kLinOneThreads)
    linear_decode_one_kernel(const LinearParams p, const int n_tiles) {
  constexpr int R = DK / (4 * RS);        // rows of a lane
  constexpr int U = R < 16 ? R : 16;      // of them loaded together
  constexpr int kTilesPerBlock = kLinOneThreads / 32 / RS;
  __shared__ float part[RS == 1 ? 1 : RS][64];
  const int warp = threadIdx.x >> 5;
  const int lane = threadIdx.x & 31;
  const int rs = warp % RS;
  const int tile = blockIdx.x * kTilesPerBlock + warp / RS;
  if (tile >= n_tiles) return;  // whole warps; with RS > 1 the whole block
  const int cols = p.D_v / 64;
  const int ct = tile % cols;
  const int bh = tile / cols;
  const int h = bh % p.H_v;
  const int b = bh / p.H_v;
  const int cg = lane & 7, rl = lane >> 3;
  uint16_t* out = p.out + static_cast<size_t>(bh) * p.D_v + ct * 64;

  int s, L, n;
  linear_item(p, b, s, L, n);
  if (L == 0) {  // padded or skipped: +0.0, the slot untouched
    if (rs == 0 && lane < 8) reinterpret_cast<uint4*>(out)[lane] = make_uint4(0u, 0u, 0u, 0u);
    return;  // L is the same for every warp of a tile
  }
  const int row0 = rs * (DK / RS) + rl * R;
  uint16_t* state = p.state_pool +
                    ((static_cast<size_t>(s) * p.H_v + h) * DK + row0) * p.D_v + ct * 64 + cg * 8;
  uint4 w[U];
#pragma unroll
  for (int i = 0; i < U; ++i)
    w[i] = *reinterpret_cast<const uint4*>(state + static_cast<size_t>(i) * p.D_v);
  const size_t qk = (static_cast<size_t>(b) * p.H_qk + h / p.group) * DK + row0;
  float v[8];
  load_bf16<8>(p.value + static_cast<size_t>(bh) * p.D_v + ct * 64 + cg * 8, v);
  const float lambda = decay_power(p.log_decay[h], 1);
  unsigned long long v2[4], o2[4];
  const unsigned long long l2 = pk(lambda, lambda);
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    v2[e] = pk(v[2 * e], v[2 * e + 1]);
    o2[e] = 0ull;
  }
#pragma unroll
  for (int i0 = 0; i0 < R; i0 += U) {
    float kf[U], qf[U];
    load_bf16<U>(p.key + qk + i0, kf);
    load_bf16<U>(p.query + qk + i0, qf);
#pragma unroll
    for (int i = 0; i < U; ++i) {
      const uint32_t x[4] = {w[i].x, w[i].y, w[i].z, w[i].w};
      if (i0 + U < R)  // the next rows' loads take the register that is now free
        w[i] = *reinterpret_cast<const uint4*>(state + static_cast<size_t>(i0 + U + i) * p.D_v);
      const unsigned long long k2 = pk(kf[i], kf[i]), q2 = pk(qf[i], qf[i]);
      uint32_t y[4];
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const unsigned long long s2 =
            fma2(k2, v2[e], mul2(l2, pk(bf16_lo(x[e]), bf16_hi(x[e]))));
        o2[e] = fma2(q2, s2, o2[e]);
        const float2 f = upk(s2);
        y[e] = pack_bf16x2(f.x, f.y);
      }
      if (n > 0)
        *reinterpret_cast<uint4*>(state + static_cast<size_t>(i0 + i) * p.D_v) =
            make_uint4(y[0], y[1], y[2], y[3]);
    }
  }
  float o[8];
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    const float2 f = upk(o2[e]);
    o[2 * e] = f.x;
    o[2 * e + 1] = f.y;
  }
#pragma unroll
  for (int e = 0; e < 8; ++e) {
    o[e] += __shfl_xor_sync(0xffffffffu, o[e], 8);
    o[e] += __shfl_xor_sync(0xffffffffu, o[e], 16);
  }
  if constexpr (RS == 1) {
    if (rl == 0)
      reinterpret_cast<uint4*>(out)[cg] =
          make_uint4(pack_bf16x2(o[0] * p.scale, o[1] * p.scale),
                     pack_bf16x2(o[2] * p.scale, o[3] * p.scale),
                     pack_bf16x2(o[4] * p.scale, o[5] * p.scale),
                     pack_bf16x2(o[6] * p.scale, o[7] * p.scale));
  } else {
    if (rl == 0) {
#pragma unroll
      for (int e = 0; e < 8; ++e) part[rs][cg * 8 + e] = o[e];
    }
    __syncthreads();
    if (threadIdx.x < 32) {
      float a = 0.0f, c = 0.0f;
#pragma unroll
      for (int r = 0; r < RS; ++r) {
        a += part[r][2 * lane];
        c += part[r][2 * lane + 1];
      }
      reinterpret_cast<uint32_t*>(out)[lane] = pack_bf16x2(a * p.scale, c * p.scale);
    }
  }
}

// ---------------------------------------------------------------- several tokens

// A block owns one (item, value head); each of its warps takes tiles of 32
// columns: 8 lanes of 4 columns by 4 row groups, and all D_k rows.
constexpr int kLinManyMaxThreads = 256;
constexpr int kLinManyAhead = 8;  // rows of a lane in flight

// Shared memory of a block: per row the L <= 8 queries and the 8 weighted
// keys as fp32 (token-contiguous, so a pair of tokens is one 64-bit operand),
// and the 8 x 8 products lambda^{t-s} q_t.k_s.
template <int DK>
struct LinManyShared {
  float q[DK][8];
  float k[DK][8];
  float a[8][8];
};

// Columns [col, col + 4) of a lane for L tokens, NP = ceil(L / 2) pairs.
template <int DK, int NP>
__device__ __forceinline__ void linear_many_tile(const LinearParams& p,
                                                 const LinManyShared<DK>& sh, uint16_t* state,
                                                 const uint16_t* value, uint16_t* out, int L,
                                                 int n, float lambda_n, float log_decay, int rl) {
  constexpr int R = DK / 4;
  constexpr int U = kLinManyAhead;
  const size_t stride = p.D_v;
  uint2 w[U];
#pragma unroll
  for (int i = 0; i < U; ++i) w[i] = *reinterpret_cast<const uint2*>(state + i * stride);
  // v of the committed tokens as pairs per column. A token that is not
  // committed has weight 0, but its value may be infinite: it is not read here.
  unsigned long long v2[NP][4], o2[NP][4];
#pragma unroll
  for (int t = 0; t < NP; ++t) {
    float a[4] = {0.0f, 0.0f, 0.0f, 0.0f}, c[4] = {0.0f, 0.0f, 0.0f, 0.0f};
    if (2 * t < n) load_bf16<4>(value + 2 * t * stride, a);
    if (2 * t + 1 < n) load_bf16<4>(value + (2 * t + 1) * stride, c);
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      v2[t][e] = pk(a[e], c[e]);
      o2[t][e] = 0ull;
    }
  }
#pragma unroll 1
  for (int i0 = 0; i0 < R; i0 += U) {
#pragma unroll
    for (int i = 0; i < U; ++i) {
      const uint32_t x[2] = {w[i].x, w[i].y};
      if (i0 + U < R)
        w[i] = *reinterpret_cast<const uint2*>(state + (i0 + U + i) * stride);
      const int row = rl * R + i0 + i;
      const ulonglong2* qr = reinterpret_cast<const ulonglong2*>(sh.q[row]);
      const ulonglong2* kr = reinterpret_cast<const ulonglong2*>(sh.k[row]);
      unsigned long long q2[NP + 1], k2[NP + 1];
#pragma unroll
      for (int t = 0; t < NP; t += 2) {
        const ulonglong2 a = qr[t / 2], c = kr[t / 2];
        q2[t] = a.x;
        q2[t + 1] = a.y;
        k2[t] = c.x;
        k2[t + 1] = c.y;
      }
      float y[4];
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const float f = (e & 1) ? bf16_hi(x[e >> 1]) : bf16_lo(x[e >> 1]);
        const unsigned long long f2 = pk(f, f);
        unsigned long long acc = pk(lambda_n * f, 0.0f);
#pragma unroll
        for (int t = 0; t < NP; ++t) {
          o2[t][e] = fma2(q2[t], f2, o2[t][e]);
          acc = fma2(k2[t], v2[t][e], acc);
        }
        const float2 r = upk(acc);
        y[e] = r.x + r.y;
      }
      if (n > 0)
        *reinterpret_cast<uint2*>(state + (i0 + i) * stride) =
            make_uint2(pack_bf16x2(y[0], y[1]), pack_bf16x2(y[2], y[3]));
    }
  }
  // the four row groups' sums, then the tokens' own terms
#pragma unroll
  for (int t = 0; t < NP; ++t) {
    float o[2][4];
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const float2 f = upk(o2[t][e]);
      o[0][e] = f.x;
      o[1][e] = f.y;
    }
#pragma unroll
    for (int j = 0; j < 2; ++j) {
      const int tok = 2 * t + j;
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        o[j][e] += __shfl_xor_sync(0xffffffffu, o[j][e], 8);
        o[j][e] += __shfl_xor_sync(0xffffffffu, o[j][e], 16);
      }
      if (tok < L && rl == (tok & 3)) {
        const float decay = decay_power(log_decay, tok + 1);
#pragma unroll
        for (int e = 0; e < 4; ++e) o[j][e] *= decay;
        for (int u = 0; u <= tok; ++u) {  // no token after tok is read
          float v[4];
          load_bf16<4>(value + u * stride, v);
          const float c = sh.a[tok][u];
#pragma unroll
          for (int e = 0; e < 4; ++e) o[j][e] = fmaf(c, v[e], o[j][e]);
        }
        *reinterpret_cast<uint2*>(out + tok * stride) =
            make_uint2(pack_bf16x2(o[j][0] * p.scale, o[j][1] * p.scale),
                       pack_bf16x2(o[j][2] * p.scale, o[j][3] * p.scale));
      }
    }
  }
}

template <int DK>
__global__ void __launch_bounds__(kLinManyMaxThreads)
    linear_decode_many_kernel(const LinearParams p) {
  __shared__ __align__(16) LinManyShared<DK> sh;
  const int h = blockIdx.x % p.H_v;
  const int b = blockIdx.x / p.H_v;
  const int tid = threadIdx.x;
  const int warp = tid >> 5, lane = tid & 31;
  const int n_warps = blockDim.x >> 5;
  const int T = p.T;
  int s, L, n;
  linear_item(p, b, s, L, n);
  const size_t bh = static_cast<size_t>(b) * p.H_v + h;
  uint16_t* out = p.out + bh * T * p.D_v;
  // padded tokens (every token of an empty or skipped item): +0.0
  for (int e = L * (p.D_v / 8) + tid; e < T * (p.D_v / 8); e += blockDim.x)
    reinterpret_cast<uint4*>(out)[e] = make_uint4(0u, 0u, 0u, 0u);
  if (L == 0) return;

  const float log_decay = p.log_decay[h];
  const size_t qk = (static_cast<size_t>(b) * p.H_qk + h / p.group) * T * DK;
  for (int e = tid; e < 8 * DK; e += blockDim.x) {
    const int t = e / DK, i = e % DK;
    float q = 0.0f, k = 0.0f;
    if (t < L) {
      q = bf16_bits_to_f32(p.query[qk + e]);
      k = bf16_bits_to_f32(p.key[qk + e]);
    }
    sh.q[i][t] = q;
    sh.k[i][t] = k;
  }
  __syncthreads();
  // lambda^{t-s} q_t . k_s for s <= t < L, a warp a product
  for (int e = warp; e < L * L; e += n_warps) {
    const int t = e / L, u = e % L;
    if (u > t) continue;
    float d = 0.0f;
#pragma unroll
    for (int i = 0; i < DK / 32; ++i)
      d = fmaf(sh.q[lane + 32 * i][t], sh.k[lane + 32 * i][u], d);
    d = warp_sum(d);
    if (lane == 0) sh.a[t][u] = d * decay_power(log_decay, t - u);
  }
  __syncthreads();
  // the keys' weights lambda^{n-1-s} of the committed tokens; the rest leave
  // the state alone
  for (int e = tid; e < 8 * DK; e += blockDim.x) {
    const int t = e & 7, i = e >> 3;
    sh.k[i][t] = t < n ? sh.k[i][t] * decay_power(log_decay, n - 1 - t) : 0.0f;
  }
  __syncthreads();

  const int cg = lane & 7, rl = lane >> 3;
  const float lambda_n = decay_power(log_decay, n);
  uint16_t* slot = p.state_pool + (static_cast<size_t>(s) * p.H_v + h) * DK * p.D_v;
  for (int col = warp * 32 + cg * 4; col < p.D_v; col += n_warps * 32) {
    uint16_t* state = slot + static_cast<size_t>(rl * (DK / 4)) * p.D_v + col;
    const uint16_t* value = p.value + bh * T * p.D_v + col;
    uint16_t* o = out + col;
    switch ((L + 1) >> 1) {
      case 1: linear_many_tile<DK, 1>(p, sh, state, value, o, L, n, lambda_n, log_decay, rl); break;
      case 2: linear_many_tile<DK, 2>(p, sh, state, value, o, L, n, lambda_n, log_decay, rl); break;
      case 3: linear_many_tile<DK, 3>(p, sh, state, value, o, L, n, lambda_n, log_decay, rl); break;
      default: linear_many_tile<DK, 4>(p, sh, state, value, o, L, n, lambda_n, log_decay, rl);
    }
  }
}

}  // namespace gdr
