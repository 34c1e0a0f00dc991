// C entry points (declared in include/gdr.h) of linear attention with one
// decay per head and of the state pool's 8-bit cache: host-side argument
// checks and kernel dispatch. As in gdr_api.cu, every check runs before
// anything is queued, and device values (lengths, slots, entries, decays) are
// handled by the kernels without traps.
#include <cuda.h>
#include <cuda_runtime.h>

#include <atomic>
#include <cstdint>
#include <string>

#include "gdr.h"
#include "gdr_host.h"
#include "gdr_linear_decode.cuh"
#include "gdr_linear_plan.h"
#include "gdr_linear_prefill.cuh"
#include "gdr_state_cache.cuh"

using gdr_host::fail;

namespace {

constexpr int kMaxDevices = 64;
constexpr long long kMaxGrid = 0x7fffffffLL;

// A runtime call that failed: its status, and nothing left of the error for the
// next launch to take for its own.
int cuda_failed(const std::string& what, cudaError_t err) {
  (void)cudaGetLastError();
  return fail(GDR_ERR_CUDA, what + ": " + cudaGetErrorString(err));
}

int launched(const char* what, int kernel, int D_k, int tile_cols, int layout, int grid,
             int threads, int smem, int stages) {
  const cudaError_t err = cudaGetLastError();
  if (err != cudaSuccess)
    return cuda_failed(std::string(what) + " launch failed", err);
  gdr_host::set_last_launch(
      gdr_launch_info{kernel, D_k, tile_cols, 0, layout, grid, threads, smem, stages});
  return GDR_OK;
}

// The sizes' checks of both linear-attention entry points.
int check_linear_dims(const gdr_dims* d, int max_T) {
  if (d == nullptr) return fail(GDR_ERR_NULL, "dims is NULL");
  if (d->B < 0) return fail(GDR_ERR_DIMS, "B must be >= 0");
  if (d->T < 1) return fail(GDR_ERR_DIMS, "T must be >= 1");
  if (max_T > 0 && d->T > max_T)
    return fail(GDR_ERR_DIMS, "T must be in [1, 8] (longer calls go to prefill)");
  if (d->H_qk < 1 || d->H_v < 1) return fail(GDR_ERR_DIMS, "H_qk and H_v must be >= 1");
  if (d->H_v % d->H_qk != 0) return fail(GDR_ERR_DIMS, "H_v must be a multiple of H_qk");
  if (d->D_k < 1 || d->D_v < 1) return fail(GDR_ERR_DIMS, "D_k and D_v must be >= 1");
  if (d->pool_size < 1) return fail(GDR_ERR_DIMS, "pool_size must be >= 1");
  if (d->layout != GDR_LAYOUT_KV && d->layout != GDR_LAYOUT_VK)
    return fail(GDR_ERR_DIMS, "layout must be GDR_LAYOUT_KV or GDR_LAYOUT_VK");
  if (d->D_k != 64 && d->D_k != 128)
    return fail(GDR_ERR_UNSUPPORTED, "D_k must be 64 or 128");
  if (d->D_v % gdr::kSliceCols != 0)
    return fail(GDR_ERR_UNSUPPORTED, "D_v must be a multiple of 64");
  if (d->layout != GDR_LAYOUT_KV)
    return fail(GDR_ERR_UNSUPPORTED,
                "linear attention takes the [pool, H_v, D_k, D_v] layout only");
  // B * H_v * (D_v / 64) is the largest grid any of the kernels uses
  const long long bh = static_cast<long long>(d->B) * d->H_v;
  if (bh > kMaxGrid || bh * (d->D_v / 64) > kMaxGrid)
    return fail(GDR_ERR_DIMS, "B * H_v * D_v / 64 exceeds 2^31 - 1");
  if (static_cast<long long>(d->pool_size) * d->H_v > kMaxGrid)
    return fail(GDR_ERR_DIMS, "pool_size * H_v exceeds 2^31 - 1");
  // row strides of a TMA map stay below 2^40 bytes
  const long long wide = d->D_v > d->D_k ? d->D_v : d->D_k;
  if (static_cast<long long>(d->T) * wide >= (1LL << 38))
    return fail(GDR_ERR_DIMS, "T * D exceeds 2^38");
  return GDR_OK;
}

int check_linear_pointers(const gdr_bf16* query, const gdr_bf16* key, const gdr_bf16* value,
                          const float* log_decay, const gdr_bf16* state_pool,
                          const int32_t* asl, const int32_t* idx, const gdr_bf16* out) {
  if (!query || !key || !value || !log_decay || !state_pool || !asl || !idx || !out)
    return fail(GDR_ERR_NULL, "a required tensor pointer is NULL");
  if (!gdr_host::aligned16(query) || !gdr_host::aligned16(key) || !gdr_host::aligned16(value) ||
      !gdr_host::aligned16(state_pool) || !gdr_host::aligned16(out))
    return fail(GDR_ERR_ALIGN, "query, key, value, state_pool and out must be 16-byte aligned");
  return GDR_OK;
}

gdr::LinearParams linear_params(const gdr_dims* d, const gdr_bf16* query, const gdr_bf16* key,
                                const gdr_bf16* value, const float* log_decay,
                                gdr_bf16* state_pool, const int32_t* asl, const int32_t* idx,
                                const int32_t* nat, float scale, gdr_bf16* out) {
  gdr::LinearParams p{};
  p.query = query;
  p.key = key;
  p.value = value;
  p.log_decay = log_decay;
  p.state_pool = state_pool;
  p.out = out;
  p.seq_lengths = asl;
  p.state_indices = idx;
  p.num_accepted = nat;
  p.scale = scale;
  p.B = d->B;
  p.T = d->T;
  p.H_qk = d->H_qk;
  p.H_v = d->H_v;
  p.D_v = d->D_v;
  p.pool_size = d->pool_size;
  p.group = d->H_v / d->H_qk;
  return p;
}

// ---------------------------------------------------------------- launches

// [groups, T, D] bf16 as boxes of 64 columns x `rows` rows of one group.
int encode_rows_map(const gdr_bf16* base, int D, int T, long long groups, int rows,
                    CUtensorMap* map) {
  PFN_cuTensorMapEncodeTiled_v12000 encode = gdr_host::tensor_map_encoder();
  if (encode == nullptr) return fail(GDR_ERR_CUDA, "cuTensorMapEncodeTiled is unavailable");
  const cuuint64_t gdim[3] = {static_cast<cuuint64_t>(D), static_cast<cuuint64_t>(T),
                              static_cast<cuuint64_t>(groups)};
  const cuuint64_t gstride[2] = {static_cast<cuuint64_t>(D) * 2,
                                 static_cast<cuuint64_t>(T) * D * 2};
  const cuuint32_t box[3] = {64, static_cast<cuuint32_t>(rows), 1};
  const cuuint32_t estride[3] = {1, 1, 1};
  const CUresult cr =
      encode(map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, const_cast<gdr_bf16*>(base), gdim, gstride,
             box, estride, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
             CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
  if (cr != CUDA_SUCCESS) return fail(GDR_ERR_CUDA, "cuTensorMapEncodeTiled failed");
  return GDR_OK;
}

template <typename K>
int opt_in_smem(K kernel, int smem, const gdr_host::Device& dev, std::atomic<bool>* ready) {
  if (smem > dev.smem_optin)
    return fail(GDR_ERR_UNSUPPORTED, "prefill tile does not fit in shared memory");
  if (ready[dev.ordinal].load(std::memory_order_acquire)) return GDR_OK;
  cudaError_t err = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
  if (err == cudaSuccess)
    err = cudaFuncSetAttribute(kernel, cudaFuncAttributePreferredSharedMemoryCarveout,
                               cudaSharedmemCarveoutMaxShared);
  if (err != cudaSuccess)
    return cuda_failed("kernel attributes", err);
  ready[dev.ordinal].store(true, std::memory_order_release);
  return GDR_OK;
}

// ---------------------------------------------------------------- decode

constexpr int kLdBlocksPerSm = 4;

template <int DK>
int launch_linear_decode(const gdr::LinearParams& p, const gdr_host::Device& dev,
                         cudaStream_t stream) {
  using Shape = gdr::LdShape<DK>;
  static std::atomic<bool> ready[kMaxDevices];
  auto kernel = gdr::linear_decode_kernel<DK>;
  int rc = opt_in_smem(kernel, Shape(Shape::kMaxCols, gdr::kMaxT).smem(), dev, ready);
  CUtensorMap pool_map;
  if (rc == GDR_OK)
    rc = encode_rows_map(p.state_pool, p.D_v, DK, static_cast<long long>(p.pool_size) * p.H_v, DK,
                         &pool_map);
  if (rc != GDR_OK) return rc;
  // The widest part that still gives every SM kLdBlocksPerSm blocks, as many as run
  // on it at once. Narrower parts repeat the work on q and k: with 16 the step of 64
  // items of 32 heads, 128 x 128, takes 32.9 us against 28.8; with 1 a single item of
  // 64 heads would leave half of the SMs idle.
  const long long heads = static_cast<long long>(p.B) * p.H_v;
  int cols = Shape::kMaxCols;
  while (cols > 64 && (cols >= 2 * p.D_v ||
                       heads * ((p.D_v - 1) / cols + 1) <
                           static_cast<long long>(kLdBlocksPerSm) * dev.sms))
    cols /= 2;
  const int parts = (p.D_v - 1) / cols + 1;
  const int grid = static_cast<int>(heads) * parts;
  const int smem = Shape(cols, p.T).smem();
  gdr::LinearDecodeParams prm{};
  prm.p = p;
  prm.part_cols = cols;
  prm.parts = gdr::FastDiv::by(static_cast<uint32_t>(parts));
  prm.heads = gdr::FastDiv::by(static_cast<uint32_t>(p.H_v));
  prm.group = gdr::FastDiv::by(static_cast<uint32_t>(p.group));
  kernel<<<grid, gdr::kLdThreads, smem, stream>>>(pool_map, prm);
  return launched("linear decode", GDR_KERNEL_LINEAR_DECODE, DK, cols, GDR_LAYOUT_KV, grid,
                  gdr::kLdThreads, smem, 1);
}

// ---------------------------------------------------------------- prefill

// A launch that, with `overlap`, may start before the one ahead of it on the
// stream is done (the kernel waits for that one where it needs its results), or,
// with `together`, has all its blocks on the GPU at once (they wait for one
// another).
template <typename... P, typename... A>
cudaError_t launch_with(void (*kernel)(P...), int grid, int threads, int smem, bool overlap,
                        bool together, cudaStream_t stream, const A&... args) {
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3(static_cast<unsigned>(grid));
  cfg.blockDim = dim3(static_cast<unsigned>(threads));
  cfg.dynamicSmemBytes = static_cast<size_t>(smem);
  cfg.stream = stream;
  cudaLaunchAttribute attr{};
  if (overlap) {
    attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr.val.programmaticStreamSerializationAllowed = 1;
  } else {
    attr.id = cudaLaunchAttributeCooperative;
    attr.val.cooperative = 1;
  }
  cfg.attrs = &attr;
  cfg.numAttrs = overlap || together ? 1 : 0;
  return cudaLaunchKernelEx(&cfg, kernel, args...);
}

template <int DK>
int launch_linear_prefill(const gdr::LinearParams& p, const gdr::PrefillPlan& plan,
                          uint8_t* workspace, const gdr_host::Device& dev,
                          cudaStream_t stream) {
  using Shape = gdr::LpShape<DK>;
  using SegShape = gdr::LsShape<DK>;
  static std::atomic<bool> ready[kMaxDevices], seg_ready[kMaxDevices];
  auto kernel = gdr::linear_prefill_kernel<DK>;
  auto seg_kernel = gdr::linear_segment_kernel<DK>;
  int rc = opt_in_smem(kernel, Shape::kSmem, dev, ready);
  if (rc == GDR_OK) rc = opt_in_smem(seg_kernel, SegShape::kSmem, dev, seg_ready);
  CUtensorMap q_map, k_map, v_map, o_map, pool_map;
  const long long qk = static_cast<long long>(p.B) * p.H_qk;
  const long long vo = static_cast<long long>(p.B) * p.H_v;
  const long long slots = static_cast<long long>(p.pool_size) * p.H_v;
  constexpr int rows = gdr::kLpChunk;
  if (rc == GDR_OK) rc = encode_rows_map(p.query, DK, p.T, qk, rows, &q_map);
  if (rc == GDR_OK) rc = encode_rows_map(p.key, DK, p.T, qk, rows, &k_map);
  if (rc == GDR_OK) rc = encode_rows_map(p.value, p.D_v, p.T, vo, rows, &v_map);
  if (rc == GDR_OK) rc = encode_rows_map(p.out, p.D_v, p.T, vo, rows, &o_map);
  if (rc == GDR_OK) rc = encode_rows_map(p.state_pool, p.D_v, DK, slots, DK, &pool_map);
  if (rc != GDR_OK) return rc;
  gdr::LinearPrefillParams prm{};
  prm.p = p;
  prm.slices = plan.slices;
  prm.stream = plan.stream;
  prm.team = plan.team;
  prm.segments = plan.segments;
  prm.seg_chunks = plan.seg_chunks;
  prm.starts = reinterpret_cast<float*>(workspace);
  prm.flags = reinterpret_cast<int*>(workspace + plan.states);
  const int tiles = p.B * p.H_v * plan.slices;
  cudaError_t err = cudaSuccess;
  if (plan.stream) {
    err = cudaMemsetAsync(prm.flags, 0, static_cast<size_t>(plan.grid) * 4, stream);
  } else if (plan.segments > 1) {
    seg_kernel<<<tiles * (plan.segments - 1), gdr::kLsThreads, SegShape::kSmem, stream>>>(
        k_map, v_map, prm);
    err = cudaGetLastError();
    if (err == cudaSuccess)
      err = launch_with(gdr::linear_scan_kernel<DK>,
                        tiles * (DK * gdr::kLpCols / gdr::kLscanThreads), gdr::kLscanThreads, 0,
                        true, false, stream, prm);
  }
  if (err == cudaSuccess)
    err = launch_with(kernel, plan.grid, gdr::kLpThreads, Shape::kSmem, plan.segments > 1,
                      plan.stream, stream, q_map, k_map, v_map, o_map, pool_map, prm);
  if (err != cudaSuccess)
    return cuda_failed("linear prefill launch", err);
  return launched("linear prefill", GDR_KERNEL_LINEAR_PREFILL, DK, gdr::kLpCols, GDR_LAYOUT_KV,
                  plan.grid, gdr::kLpThreads, Shape::kSmem, Shape::kStages);
}

// ---------------------------------------------------------------- 8-bit cache

int check_cache(const void* pool, int32_t pool_size, const int32_t* slots, const void* codes,
                const float* scales, int32_t cache_size, const int32_t* entries, int32_t n,
                int64_t slot_values, int type, gdr::CacheParams* p) {
  if (n < 0) return fail(GDR_ERR_DIMS, "n must be >= 0");
  if (pool_size < 1 || cache_size < 1)
    return fail(GDR_ERR_DIMS, "pool_size and cache_size must be >= 1");
  if (slot_values < gdr::kCacheGroup || slot_values % gdr::kCacheGroup != 0)
    return fail(GDR_ERR_DIMS, "slot_values must be a positive multiple of 64");
  if (type != GDR_CACHE_INT8 && type != GDR_CACHE_E4M3)
    return fail(GDR_ERR_UNSUPPORTED, "cache type must be GDR_CACHE_INT8 or GDR_CACHE_E4M3");
  // the most blocks either form needs
  const long long blocks = (slot_values - 1) / (gdr::kCacheThreads * gdr::kCacheAheadFew * 8) + 1;
  if (blocks > kMaxGrid || blocks * n > kMaxGrid)
    return fail(GDR_ERR_DIMS, "n * slot_values / 2048 exceeds 2^31 - 1");
  const long long most = pool_size > cache_size ? pool_size : cache_size;
  if (slot_values > (1LL << 61) / most)
    return fail(GDR_ERR_DIMS, "pool or cache exceeds 2^61 values");
  if (n == 0) return GDR_OK;
  if (!pool || !slots || !codes || !scales || !entries)
    return fail(GDR_ERR_NULL, "a required tensor pointer is NULL");
  if (!gdr_host::aligned16(pool) || !gdr_host::aligned16(codes) || !gdr_host::aligned16(scales))
    return fail(GDR_ERR_ALIGN, "state_pool, cache and scales must be 16-byte aligned");
  p->pool = const_cast<uint16_t*>(static_cast<const uint16_t*>(pool));
  p->codes = const_cast<uint8_t*>(static_cast<const uint8_t*>(codes));
  p->scales = const_cast<float*>(scales);
  p->slots = slots;
  p->entries = entries;
  p->slot_values = slot_values;
  p->pool_size = pool_size;
  p->cache_size = cache_size;
  return GDR_OK;
}

// Launches the form of a cache kernel that fits the call: 8 pieces a lane where
// that still gives every SM kCacheBlocksPerSm blocks.
constexpr int kCacheBlocksPerSm = 8;
template <typename K>
int launch_cache(K many, K few, const char* what, gdr::CacheParams p, int n,
                 gdr_stream_t stream) {
  gdr_host::Device dev;
  const int rc = gdr_host::current_device(&dev);
  if (rc != GDR_OK) return rc;
  const auto blocks = [&](int ahead) {
    return (p.slot_values - 1) / (gdr::kCacheThreads * ahead * 8) + 1;
  };
  const bool is_few = blocks(gdr::kCacheAhead) * n < kCacheBlocksPerSm * dev.sms;
  p.blocks_per_slot =
      static_cast<int>(blocks(is_few ? gdr::kCacheAheadFew : gdr::kCacheAhead));
  const int grid = n * p.blocks_per_slot;
  (is_few ? few : many)<<<grid, gdr::kCacheThreads, 0, reinterpret_cast<cudaStream_t>(stream)>>>(p);
  return launched(what, GDR_KERNEL_STATE_CACHE, 0, 0, GDR_LAYOUT_KV, grid, gdr::kCacheThreads, 0,
                  0);
}

}  // namespace

namespace gdr_host {

cudaError_t linear_device_error(unsigned int* flags, bool reset) {
  cudaError_t err = cudaMemcpyFromSymbol(flags, gdr::g_device_error, sizeof(*flags));
  if (err == cudaSuccess && reset) {
    const unsigned int zero = 0;
    err = cudaMemcpyToSymbol(gdr::g_device_error, &zero, sizeof(zero));
  }
  return err;
}

#ifdef GDR_TEST_HOOKS
cudaError_t linear_set_hooks(long long wait_limit_cycles, int hold_tile) {
  cudaError_t err =
      cudaMemcpyToSymbol(gdr::g_test_wait_limit, &wait_limit_cycles, sizeof(wait_limit_cycles));
  if (err == cudaSuccess)
    err = cudaMemcpyToSymbol(gdr::g_test_hold_tile, &hold_tile, sizeof(hold_tile));
  return err;
}
#endif

}  // namespace gdr_host

extern "C" {

GDR_API int gdr_linear_attention_decode(const gdr_dims* dims, const gdr_bf16* query,
                                        const gdr_bf16* key, const gdr_bf16* value,
                                        const float* log_decay, gdr_bf16* state_pool,
                                        const int32_t* actual_seq_lengths,
                                        const int32_t* ssm_state_indices,
                                        const int32_t* num_accepted_tokens, float scale_value,
                                        gdr_bf16* out, gdr_stream_t stream) {
  gdr_host::set_last_launch(gdr_launch_info{});
  int rc = check_linear_dims(dims, gdr::kMaxT);
  if (rc != GDR_OK) return rc;
  if (dims->B == 0) return GDR_OK;
  rc = check_linear_pointers(query, key, value, log_decay, state_pool, actual_seq_lengths,
                             ssm_state_indices, out);
  if (rc != GDR_OK) return rc;
  gdr_host::Device dev;
  rc = gdr_host::current_device(&dev);
  if (rc != GDR_OK) return rc;
  const gdr::LinearParams p =
      linear_params(dims, query, key, value, log_decay, state_pool, actual_seq_lengths,
                    ssm_state_indices, num_accepted_tokens, scale_value, out);
  const cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
  return dims->D_k == 64 ? launch_linear_decode<64>(p, dev, st)
                         : launch_linear_decode<128>(p, dev, st);
}

GDR_API int gdr_linear_attention_prefill_workspace(const gdr_dims* dims, int64_t* bytes) {
  if (bytes == nullptr) return fail(GDR_ERR_NULL, "bytes is NULL");
  *bytes = 0;
  int rc = check_linear_dims(dims, 0);
  if (rc != GDR_OK || dims->B == 0) return rc;
  gdr_host::Device dev;
  rc = gdr_host::current_device(&dev);
  if (rc != GDR_OK) return rc;
  *bytes = gdr::plan_prefill(dims, dev.sms).workspace;
  return GDR_OK;
}

GDR_API int gdr_linear_attention_prefill(const gdr_dims* dims, const gdr_bf16* query,
                                         const gdr_bf16* key, const gdr_bf16* value,
                                         const float* log_decay, gdr_bf16* state_pool,
                                         const int32_t* actual_seq_lengths,
                                         const int32_t* ssm_state_indices, float scale_value,
                                         gdr_bf16* out, void* workspace, int64_t workspace_bytes,
                                         gdr_stream_t stream) {
  gdr_host::set_last_launch(gdr_launch_info{});
  int rc = check_linear_dims(dims, 0);
  if (rc != GDR_OK) return rc;
  if (dims->B == 0) return GDR_OK;
  rc = check_linear_pointers(query, key, value, log_decay, state_pool, actual_seq_lengths,
                             ssm_state_indices, out);
  if (rc != GDR_OK) return rc;
  if (!gdr_host::aligned16(workspace))
    return fail(GDR_ERR_ALIGN, "workspace must be 16-byte aligned");
  gdr_host::Device dev;
  rc = gdr_host::current_device(&dev);
  if (rc != GDR_OK) return rc;
  const gdr::PrefillPlan plan = gdr::plan_prefill(dims, dev.sms);
  const cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
  if (plan.workspace > 0 && (workspace == nullptr || workspace_bytes < plan.workspace))
    return fail(GDR_ERR_NULL, "workspace is smaller than gdr_linear_attention_prefill_workspace "
                              "asks for");
  const gdr::LinearParams p =
      linear_params(dims, query, key, value, log_decay, state_pool, actual_seq_lengths,
                    ssm_state_indices, nullptr, scale_value, out);
  // a few tokens are a decode call with all of them committed (64 items of 32
  // heads, 8 tokens, 128 x 128: 27 us against 81 us in a chunk of 128)
  if (dims->T <= gdr::kMaxT)
    return dims->D_k == 64 ? launch_linear_decode<64>(p, dev, st)
                           : launch_linear_decode<128>(p, dev, st);
  uint8_t* ws = static_cast<uint8_t*>(workspace);
  return dims->D_k == 64 ? launch_linear_prefill<64>(p, plan, ws, dev, st)
                         : launch_linear_prefill<128>(p, plan, ws, dev, st);
}

GDR_API int gdr_state_quantize(const gdr_bf16* state_pool, int32_t pool_size,
                               const int32_t* ssm_state_indices, void* cache, float* scales,
                               int32_t cache_size, const int32_t* cache_indices, int32_t n,
                               int64_t slot_values, int cache_type, gdr_stream_t stream) {
  gdr_host::set_last_launch(gdr_launch_info{});
  gdr::CacheParams p{};
  const int rc = check_cache(state_pool, pool_size, ssm_state_indices, cache, scales, cache_size,
                             cache_indices, n, slot_values, cache_type, &p);
  if (rc != GDR_OK || n == 0) return rc;
  constexpr int many = gdr::kCacheAhead, few = gdr::kCacheAheadFew;
  if (cache_type == GDR_CACHE_E4M3)
    return launch_cache(gdr::state_quantize_kernel<true, many>, gdr::state_quantize_kernel<true, few>,
                        "state quantize", p, n, stream);
  return launch_cache(gdr::state_quantize_kernel<false, many>, gdr::state_quantize_kernel<false, few>,
                      "state quantize", p, n, stream);
}

GDR_API int gdr_state_dequantize(const void* cache, const float* scales, int32_t cache_size,
                                 const int32_t* cache_indices, gdr_bf16* state_pool,
                                 int32_t pool_size, const int32_t* ssm_state_indices, int32_t n,
                                 int64_t slot_values, int cache_type, gdr_stream_t stream) {
  gdr_host::set_last_launch(gdr_launch_info{});
  gdr::CacheParams p{};
  const int rc = check_cache(state_pool, pool_size, ssm_state_indices, cache, scales, cache_size,
                             cache_indices, n, slot_values, cache_type, &p);
  if (rc != GDR_OK || n == 0) return rc;
  constexpr int many = gdr::kCacheAhead, few = gdr::kCacheAheadFew;
  if (cache_type == GDR_CACHE_E4M3)
    return launch_cache(gdr::state_dequantize_kernel<true, many>, gdr::state_dequantize_kernel<true, few>,
                        "state dequantize", p, n, stream);
  return launch_cache(gdr::state_dequantize_kernel<false, many>, gdr::state_dequantize_kernel<false, few>,
                      "state dequantize", p, n, stream);
}

}  // extern "C"
