// Launch parameters shared by the linear-attention kernels (one decay per
// head, no delta rule):
//   S_t = lambda_h S_{t-1} + k_t v_t^T,  lambda_h = exp(log_decay_h)
//   o_t = scale * S_t^T q_t
// and the powers of lambda they use.
#pragma once

#include <cuda_runtime.h>
#include <stdint.h>

#include "gdr_decode.cuh"

namespace gdr {

struct LinearParams {
  const uint16_t* query;         // [B, H_qk, T, D_k] bf16
  const uint16_t* key;           // [B, H_qk, T, D_k] bf16
  const uint16_t* value;         // [B, H_v, T, D_v] bf16
  const float* log_decay;        // [H_v] fp32
  uint16_t* state_pool;          // [pool, H_v, D_k, D_v] bf16, in place
  uint16_t* out;                 // [B, H_v, T, D_v] bf16
  const int32_t* seq_lengths;    // [B]
  const int32_t* state_indices;  // [B]
  const int32_t* num_accepted;   // [B] or NULL (decode only)
  float scale;
  int B, T, H_qk, H_v, D_v, pool_size;
  int group;  // H_v / H_qk
};

// lambda^n = exp(n log_decay). n = 0 gives 1 for every log_decay, -inf
// (a head that forgets at once) included.
__device__ __forceinline__ float decay_power(float log_decay, int n) {
  return n == 0 ? 1.0f : expf(log_decay * static_cast<float>(n));
}

// Item b's slot s, valid tokens L (0 when the slot is outside the pool) and
// committed tokens n.
__host__ __device__ __forceinline__ void linear_item(const LinearParams& p, int b, int& s,
                                                     int& L, int& n) {
  s = p.state_indices[b];
  L = p.seq_lengths[b];
  L = L < 0 ? 0 : (L > p.T ? p.T : L);
  if (s < 0 || s >= p.pool_size) L = 0;
  n = p.num_accepted != nullptr ? p.num_accepted[b] : L;
  n = n < 0 ? 0 : (n > L ? L : n);
}

// 8 x 8 matrices of 16-bit values between shared memory and registers, four (or
// two) at a time; lane i gives the address of row i % 8 of matrix i / 8.
__device__ __forceinline__ void ldmatrix_x4(uint32_t addr, uint32_t (&r)[4]) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0, %1, %2, %3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr)
               : "memory");
}
__device__ __forceinline__ void ldmatrix_x4_trans(uint32_t addr, uint32_t (&r)[4]) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0, %1, %2, %3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr)
               : "memory");
}
__device__ __forceinline__ void ldmatrix_x2_trans(uint32_t addr, uint32_t (&r)[2]) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x2.trans.shared.b16 {%0, %1}, [%2];"
               : "=r"(r[0]), "=r"(r[1])
               : "r"(addr)
               : "memory");
}
__device__ __forceinline__ void stmatrix_x4(uint32_t addr, const uint32_t (&r)[4]) {
  asm volatile("stmatrix.sync.aligned.m8n8.x4.shared.b16 [%0], {%1, %2, %3, %4};" ::"r"(addr),
               "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3])
               : "memory");
}
__device__ __forceinline__ void stmatrix_x4_trans(uint32_t addr, const uint32_t (&r)[4]) {
  asm volatile("stmatrix.sync.aligned.m8n8.x4.trans.shared.b16 [%0], {%1, %2, %3, %4};" ::"r"(addr),
               "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3])
               : "memory");
}

}  // namespace gdr
