// The state pool's 8-bit cache: whole slots written to cache entries as codes
// with one fp32 scale for each 64 consecutive values, and read back into
// slots.
//
//   m     = max |x| of the group
//   scale = m / top, factor = top / m    (top = 127 for int8, 448 for e4m3)
//   code  = round to nearest even of x * factor
//   x'    = bf16(code * scale)
// A group with m < 2^-100 is held as zeros (top / m would overflow further
// down). A group with an infinity or a NaN gets scale = NaN, so that all of it
// reads back as NaN: what was not a number never comes back as one.
//
// Both kernels move 2 + 1 + 4/64 bytes a value and do little with it, so HBM
// bounds them: 16 bytes a lane and access, and each block one contiguous piece
// of one slot (a slot is contiguous whatever its layout, and rows are whole
// groups in both layouts of the pool). A lane has 8 accesses in flight, 128
// threads a block: 256 of 512 slots of 64 heads of 64 x 512 written and read
// back in 500 to 542 us by the GPU (6.1 to 6.6 TB/s, the copy rate; 4 in flight and
// 256 threads 521 us where this took 500). Calls too small
// to fill the SMs that way take 2 accesses a lane and four times the blocks: one
// such slot, 8.4 us for both calls against 10.5 us.
#pragma once

#include <cuda_fp16.h>
#include <cuda_fp8.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include "gdr_decode.cuh"

namespace gdr {

constexpr int kCacheGroup = 64;        // values that share a scale
constexpr int kCacheThreads = 128;
constexpr int kCacheAhead = 8, kCacheAheadFew = 2;  // 8-value pieces a lane takes at once
constexpr float kCacheFloor = 7.888609052210118e-31f;  // 2^-100

struct CacheParams {
  uint16_t* pool;         // [pool, slot_values] bf16
  uint8_t* codes;         // [entries, slot_values]
  float* scales;          // [entries, slot_values / 64]
  const int32_t* slots;   // [n]
  const int32_t* entries; // [n]
  int64_t slot_values;
  int pool_size, cache_size;
  int blocks_per_slot;
};

// Slot and entry of this block's pair, its first value; false when either
// index is outside its range (the pair is skipped).
__device__ __forceinline__ bool cache_pair(const CacheParams& p, int64_t* slot, int64_t* entry,
                                           int64_t* first, int per_block) {
  const int i = blockIdx.x / p.blocks_per_slot;
  *slot = p.slots[i];
  *entry = p.entries[i];
  *first = static_cast<int64_t>(blockIdx.x % p.blocks_per_slot) * per_block;
  return *slot >= 0 && *slot < p.pool_size && *entry >= 0 && *entry < p.cache_size;
}

__device__ __forceinline__ uint32_t max_u16x2(uint32_t a, uint32_t b) { return __vmaxu2(a, b); }

// Four values (already times the factor) as four codes, first in the low byte.
template <bool E4M3>
__device__ __forceinline__ uint32_t pack_codes(float a, float b, float c, float d) {
  if constexpr (E4M3) {
    uint16_t lo, hi;
    asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(lo) : "f"(b), "f"(a));
    asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(hi) : "f"(d), "f"(c));
    return static_cast<uint32_t>(lo) | (static_cast<uint32_t>(hi) << 16);
  } else {
    // 1.5 * 2^23 + y: the sum rounds y to an integer, to nearest even, and its
    // low byte is that integer in two's complement
    const float magic = 12582912.0f;
    const uint32_t x = __float_as_uint(__fadd_rn(a, magic));
    const uint32_t y = __float_as_uint(__fadd_rn(b, magic));
    const uint32_t z = __float_as_uint(__fadd_rn(c, magic));
    const uint32_t w = __float_as_uint(__fadd_rn(d, magic));
    return __byte_perm(__byte_perm(x, y, 0x0040), __byte_perm(z, w, 0x0040), 0x5410);
  }
}

// Four codes as fp32 (exact).
template <bool E4M3>
__device__ __forceinline__ void unpack_codes(uint32_t w, float (&f)[4]) {
  if constexpr (E4M3) {
    uint32_t lo, hi;
    asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(lo) : "h"(static_cast<uint16_t>(w)));
    asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(hi) : "h"(static_cast<uint16_t>(w >> 16)));
    const float2 a = __half22float2(*reinterpret_cast<const __half2*>(&lo));
    const float2 b = __half22float2(*reinterpret_cast<const __half2*>(&hi));
    f[0] = a.x;
    f[1] = a.y;
    f[2] = b.x;
    f[3] = b.y;
  } else {
    // byte + 128 in the low bits of 2^23, minus 2^23 + 128
    const uint32_t u = w ^ 0x80808080u;
#pragma unroll
    for (int e = 0; e < 4; ++e)
      f[e] = __uint_as_float(__byte_perm(u, 0x4B000000u, 0x7440 + e)) - 8388736.0f;
  }
}

// A block takes kCacheThreads * AHEAD pieces of 8 values; 8 lanes share a group.
template <bool E4M3, int AHEAD>
__global__ void __launch_bounds__(kCacheThreads) state_quantize_kernel(const CacheParams p) {
  constexpr float top = E4M3 ? 448.0f : 127.0f;
  int64_t slot, entry, first;
  if (!cache_pair(p, &slot, &entry, &first, kCacheThreads * AHEAD * 8)) return;
  const uint16_t* src = p.pool + slot * p.slot_values;
  uint8_t* dst = p.codes + entry * p.slot_values;
  float* sdst = p.scales + entry * (p.slot_values / kCacheGroup);
  uint4 w[AHEAD];
  int64_t at[AHEAD];
#pragma unroll
  for (int u = 0; u < AHEAD; ++u) {
    at[u] = first + (u * kCacheThreads + threadIdx.x) * 8;
    w[u] = make_uint4(0u, 0u, 0u, 0u);
    // a slot is whole groups, so the 8 lanes of a group agree
    if (at[u] < p.slot_values) w[u] = *reinterpret_cast<const uint4*>(src + at[u]);
  }
#pragma unroll
  for (int u = 0; u < AHEAD; ++u) {
    const uint32_t x[4] = {w[u].x, w[u].y, w[u].z, w[u].w};
    // magnitudes as integers: their order is the values', with inf and NaN on top
    uint32_t m = max_u16x2(max_u16x2(x[0] & 0x7fff7fffu, x[1] & 0x7fff7fffu),
                           max_u16x2(x[2] & 0x7fff7fffu, x[3] & 0x7fff7fffu));
#pragma unroll
    for (int o = 1; o < 8; o <<= 1) m = max_u16x2(m, __shfl_xor_sync(0xffffffffu, m, o));
    const uint32_t mb = (m >> 16) > (m & 0xffffu) ? (m >> 16) : (m & 0xffffu);
    const float most = __uint_as_float(mb << 16);
    float scale = 0.0f, factor = 0.0f;
    if (mb >= 0x7f80u) {
      scale = __int_as_float(0x7fffffff);
    } else if (most >= kCacheFloor) {
      scale = __fdiv_rn(most, top);
      factor = __fdiv_rn(top, most);
    }
    float y[8];
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      y[2 * e] = __fmul_rn(bf16_lo(x[e]), factor);
      y[2 * e + 1] = __fmul_rn(bf16_hi(x[e]), factor);
    }
    if (at[u] < p.slot_values) {
      *reinterpret_cast<uint2*>(dst + at[u]) =
          make_uint2(pack_codes<E4M3>(y[0], y[1], y[2], y[3]),
                     pack_codes<E4M3>(y[4], y[5], y[6], y[7]));
      if ((threadIdx.x & 7) == 0) sdst[at[u] / kCacheGroup] = scale;
    }
  }
}

template <bool E4M3, int AHEAD>
__global__ void __launch_bounds__(kCacheThreads) state_dequantize_kernel(const CacheParams p) {
  int64_t slot, entry, first;
  if (!cache_pair(p, &slot, &entry, &first, kCacheThreads * AHEAD * 8)) return;
  uint16_t* dst = p.pool + slot * p.slot_values;
  const uint8_t* src = p.codes + entry * p.slot_values;
  const float* ssrc = p.scales + entry * (p.slot_values / kCacheGroup);
  uint2 w[AHEAD];
  float scale[AHEAD];
  int64_t at[AHEAD];
#pragma unroll
  for (int u = 0; u < AHEAD; ++u) {
    at[u] = first + (u * kCacheThreads + threadIdx.x) * 8;
    if (at[u] < p.slot_values) {
      w[u] = *reinterpret_cast<const uint2*>(src + at[u]);
      scale[u] = ssrc[at[u] / kCacheGroup];
    }
  }
#pragma unroll
  for (int u = 0; u < AHEAD; ++u) {
    if (at[u] >= p.slot_values) break;
    float f[8], g[4];
    unpack_codes<E4M3>(w[u].x, g);
#pragma unroll
    for (int e = 0; e < 4; ++e) f[e] = __fmul_rn(g[e], scale[u]);
    unpack_codes<E4M3>(w[u].y, g);
#pragma unroll
    for (int e = 0; e < 4; ++e) f[4 + e] = __fmul_rn(g[e], scale[u]);
    *reinterpret_cast<uint4*>(dst + at[u]) =
        make_uint4(pack_bf16x2(f[0], f[1]), pack_bf16x2(f[2], f[3]), pack_bf16x2(f[4], f[5]),
                   pack_bf16x2(f[6], f[7]));
  }
}

}  // namespace gdr
