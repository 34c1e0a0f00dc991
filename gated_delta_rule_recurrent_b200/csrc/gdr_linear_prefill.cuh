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
// A CTA works on a tile, (item, value head, 128 columns of D_v), a chunk after
// the other. TMEM (512 columns, fp32): P | S^T q | P V | the state, transposed
// (lane = a column j of S). Roles, one warp each for the first four and one group
// of four warps for the others:
//   load     TMA of the chunk's q, k, v into a ring of stages;
//   mma      the four products: P = q k^T; S^T q; S += (V^T)(weighted k);
//            P V with P read from TMEM;
//   walk     which chunks come next (LpWalk), for all roles;
//   padding  zeros for the output rows behind the items' last tokens;
//   P        P out of TMEM, times lambda^{i-j}, masked, back as bf16 over
//            itself;
//   out      (S^T q) lambda^{i+1} to where P V is then added to it; their sum,
//            scaled, to bf16 in the chunk's v stage (both products have read v by
//            then), TMA store;
//   state    k in place times lambda^{C-1-j}; then S out of TMEM to a pair of
//            bf16 tiles (S_hi, and S_lo = S - S_hi, which takes the place of
//            the chunk's k) for the next chunk's S^T q, and back scaled by
//            lambda^C for the next chunk's sum.
// The mma warp issues the next chunk's q k^T right behind this chunk's P V, so
// the tensor pipe waits only where the chain through the state is longer.
//
// Roundings to bf16, next to the fp32 sums: P and the weighted k, since the
// other operand of their products is bf16 and one MMA takes one type. Each is
// at most 2^-8 of its term, with a random sign, about what the bf16 output's own
// rounding adds; with one of them behind each output the error is 1.4 times
// that of the output's rounding alone. The state stays fp32 from the first
// chunk to the last, and S^T q reads 16 significant bits of it.
//
// Many tiles: lengths differ, and tiles rarely fill the last wave of SMs, so with
// more tiles than SMs every SM takes an equal share of all chunks instead of whole
// tiles (8 items of 32 heads, up to 2048 tokens, 128 x 128: 94 us against 100 at the
// step that brought it). A tile that goes on in the next share hands its state to that
// CTA; a CTA hands its own on before it waits for another one's, so that only the
// chunks of one tile follow one another (128 x 128: 150 heads of 8192 tokens, 64
// chunks each, 207 us against 654 with the state held back until then; one prompt of
// 16384 tokens among seven of 256, 32 heads, 430 us against 4019: 128 chunks in a row).
// Long prompts of few heads: the chunks of a tile are cut into segments of a CTA
// each, where that is faster. A first pass sums each segment's
// sum_j lambda^{end-1-j} k_j v_j^T (half the operands, one product a chunk, no
// chain), a small scan turns those into the segments' first states, and the main
// kernel starts each segment from its own.
//
// What bounds it: a chunk takes about 4500 cycles (2.5 us; 10 us a call and 1.5 us
// a further tile of an SM besides; 3.0 us with all SMs at it). Its MMAs take 2600 of them and
// keep shared memory, where their operands are, about as busy, and three loops
// are each nearly as long: through the state (its sum, to bf16 tiles, S^T q),
// through the stage (S^T q, the next load into S_lo's place, q k^T) and through P
// (q k^T, P, P V). Skipping the work of any one of them gains 1 to 5 %. Measured:
// the call above 84 to 104 us by the draw of its lengths (350 MB in 93 us, 3.8 TB/s);
// 4 items of 16 heads, up to 4001 tokens, 64 x 512, 117 to 139 us (4.2 TB/s); one item
// of 8 heads and 32768 tokens 93 to 96 us (2.8 TB/s), of which the first pass is 28
// (alone, with cold caches).
// The loops are kept short in code as well: with all of them unrolled the roles
// together outgrew the instruction caches (144 us against 103 for the same call).
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
constexpr int kLpItems = 256;              // items whose chunks a CTA counts, at most
constexpr int kLpRegsFew = 56, kLpRegsMany = 152;  // 128 * 56 + 384 * 152 = 65536
constexpr int kLpBox = kLpChunk * 128;     // bytes of 128 rows x 64 bf16
constexpr int kLpTmemCols = 512;
constexpr int kLpTmemP = 0, kLpTmemInter = 128, kLpTmemIntra = 256, kLpTmemState = 384;
constexpr int kLpBars = 11;                // besides six per stage and two per work entry
constexpr int kLpWorks = 4;                // work entries in the ring
constexpr int kLpReaders = 14;             // warps that read them

template <int DK>
struct LpShape {
  static constexpr int kBoxes = DK / 64;                  // 64-column boxes of q and of k
  static constexpr int kStages = DK == 128 ? 2 : 3;
  static constexpr int kStageBytes = (2 * kBoxes + 2) * kLpBox;  // q, k, v
  static constexpr int kStateOff = kStages * kStageBytes;        // bf16 S^T, [128 j][DK]
  static constexpr int kBarOff = kStateOff + kBoxes * kLpBox;
  static constexpr int kPowOff = kBarOff + 8 * (6 * kStages + kLpBars + 2 * kLpWorks) + 16;
  static constexpr int kWorkOff = (kPowOff + 4 * 32 + 15) / 16 * 16;
  static constexpr int kLenOff = kWorkOff + 64 * kLpWorks;
  static constexpr int kSmem = 1024 + kLenOff + 4 * (kLpItems + 1);
  static_assert(kStageBytes % 1024 == 0 && kStateOff % 1024 == 0 && kBarOff % 8 == 0 &&
                    kPowOff % 4 == 0 && kWorkOff % 16 == 0 && kLenOff % 4 == 0,
                "alignment of what lies there");
  static_assert(kSmem <= 232448, "shared memory of a block");
};

struct LinearPrefillParams {
  LinearParams p;
  int slices;      // ceil(D_v / 128)
  int stream;      // nonzero: every team of CTAs takes an equal share of all chunks
  int team;        // CTAs of a team: that many consecutive tiles read the same q and k
  int segments;    // of a tile (1: not cut), with stream = 0
  int seg_chunks;  // chunks of a segment
  // States between CTAs, [D_k / 4][128 columns][4 rows] each (four rows of a column
  // are one 16-byte access, coalesced over the columns). With segments
  // [tiles][segments]: entry g >= 1 is the sum of segment g - 1 after the first
  // pass, and every entry the first state of its segment after the scan (of items of
  // several segments). With stream [CTAs]: what CTA c hands to CTA c + team, which may
  // read it once flags[c] is set.
  float* starts;
  // With stream [CTAs], see above. With segments [tiles][segments]: entry g >= 1 says
  // whether the first pass got to the end of the sum of segment g - 1.
  int* flags;
};

// One stretch of chunks of one tile: n chunks from chunk c0 of (item b, value
// head h, columns col0 ..), L tokens from there to the item's end. n = 0 ends
// the CTA's work.
struct alignas(16) LpWork {
  int bh, h, qk, col0;        // qk: item and query head
  int cols, slot_row, c0, n;  // slot_row: slot and value head
  int L, whole_start, whole_end;  // from the slot's state; to the slot
  float log_decay;
  int rest;  // where the walk goes on (LpWalk::hi)
};
static_assert(sizeof(LpWork) <= 64, "an entry of the ring");

// The stretches of a CTA in their order. One warp walks them and passes them on
// to the others through a ring in shared memory, ahead of time (each role doing
// it for itself cost 4000 cycles a stretch, most of them for fetching code that
// runs once a stretch).
//   stream = 0: one, segment blockIdx.x % segments of tile blockIdx.x / segments.
//   stream = 1: `team` consecutive tiles, which read the same q and k, are a unit,
//     and a team of as many CTAs takes a share [lo, hi) of the chunks in the order
//     of the units, each CTA its tile of a unit: they run side by side, and q and k
//     come from HBM once for all of them. The last unit comes first: one that goes
//     on in the next team's share hands its states over early, and one that began
//     in the share before comes last, when those have long been there.
// Callable on the host as well, where the schedule is checked without a GPU.
struct LpWalk {
  const LinearPrefillParams& prm;
  const int* before;  // stream: chunks of all items ahead of item b
  int block;          // blockIdx.x
  int lo, hi;
  // The CTA's range [lo, hi): of all teams' `all` chunks (stream), or of the chunks
  // of its tile, whose item has L tokens.
  __host__ __device__ __forceinline__ void share(int all, int teams) {
    // equal shares; only the last teams' may be short or empty, so that no empty
    // one stands between two parts of a unit
    const int each = (all - 1) / teams + 1;
    const long long from = static_cast<long long>(each) * (block / prm.team);
    lo = from < all ? static_cast<int>(from) : all;
    hi = from + each < all ? static_cast<int>(from) + each : all;
  }
  __host__ __device__ __forceinline__ void segment(int L) {
    const int chunks = (L + kLpChunk - 1) / kLpChunk;
    lo = block % prm.segments * prm.seg_chunks;
    hi = lo + prm.seg_chunks < chunks ? lo + prm.seg_chunks : chunks;
  }
  __host__ __device__ __forceinline__ void next(LpWork& w) {
    w.n = 0;
    if (hi <= lo) return;
    const LinearParams& p = prm.p;
    int tile, chunks;
    if (prm.stream) {
      const int per_item = p.H_v * prm.slices / prm.team;
      int b0 = 0, b1 = p.B - 1;  // the item of chunk hi - 1
      while (b0 < b1) {
        const int m = (b0 + b1 + 1) >> 1;
        if (before[m] < hi) {
          b0 = m;
        } else {
          b1 = m - 1;
        }
      }
      chunks = (before[b0 + 1] - before[b0]) / per_item;
      const int in_item = (hi - 1 - before[b0]) / chunks;
      const int first = before[b0] + in_item * chunks;
      tile = (b0 * per_item + in_item) * prm.team + block % prm.team;
      w.c0 = lo > first ? lo - first : 0;
      w.n = hi - first - w.c0;
      hi = first + w.c0;
    } else {
      tile = block / prm.segments;
      w.c0 = lo;
      w.n = hi - lo;
      hi = lo;
    }
    w.bh = tile / prm.slices;
    const int b = w.bh / p.H_v;
    w.h = w.bh - b * p.H_v;
    w.qk = b * p.H_qk + w.h / p.group;
    w.col0 = (tile - w.bh * prm.slices) * kLpCols;
    w.cols = p.D_v - w.col0 < kLpCols ? p.D_v - w.col0 : kLpCols;  // 64 or 128
    int s, L, n;
    linear_item(p, b, s, L, n);
    w.slot_row = s * p.H_v + w.h;
    w.L = L - w.c0 * kLpChunk;
    w.whole_end = w.n * kLpChunk >= w.L;
    // nothing orders the load of a slot by a tile's first segment and the store by its
    // last one: several segments all start from the scan's results
    w.whole_start = w.c0 == 0 && (prm.segments == 1 || w.whole_end);
    w.log_decay = p.log_decay[w.h];
    w.rest = hi;
  }
};

// Byte offset of 16-byte chunk c (8 bf16) of row r in a [128 rows][64 columns]
// box with the 128-byte swizzle.
__device__ __forceinline__ int lp_swz(int r, int c) {
  return (r * 128 + ((r & 7) << 4)) ^ (c << 4);
}

// Move registers between warpgroups (every warp of the group executes it).
template <int N>
__device__ __forceinline__ void lp_regs_dec() {
  asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(N));
}
template <int N>
__device__ __forceinline__ void lp_regs_inc() {
  asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(N));
}

// Until the launch before this one is done and its writes are visible (no
// effect on a launch that does not overlap with the one before).
__device__ __forceinline__ void lp_grid_wait() {
  asm volatile("griddepcontrol.wait;" ::: "memory");
}
__device__ __forceinline__ void lp_grid_launch_next() {
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
}

// Row r of a chunk's k times `weight`, in place. The
// weight is a pair of bf16, w = hi + lo, and k w = k hi + (k lo) one fused bf16
// operation behind a small product: the rounding of k w itself, and 2^-17 of
// it, at half the instructions of the way through fp32. With the swizzle, 8
// lanes (8 rows) touch 8 different groups of banks.
template <int kBoxes>
__device__ __forceinline__ void lp_weight_row(uint8_t* k_s, int r, float weight) {
  const __nv_bfloat16 hi = __float2bfloat16_rn(weight);
  const __nv_bfloat16 lo = __float2bfloat16_rn(weight - __bfloat162float(hi));
  const __nv_bfloat162 hi2 = __halves2bfloat162(hi, hi), lo2 = __halves2bfloat162(lo, lo);
#pragma unroll 1
  for (int x = 0; x < kBoxes; ++x) {
    uint4 w[8];
#pragma unroll
    for (int c = 0; c < 8; ++c)
      w[c] = *reinterpret_cast<const uint4*>(k_s + x * kLpBox + lp_swz(r, c));
#pragma unroll
    for (int c = 0; c < 8; ++c) {
      uint32_t y[4] = {w[c].x, w[c].y, w[c].z, w[c].w};
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const __nv_bfloat162 k2 = *reinterpret_cast<const __nv_bfloat162*>(&y[e]);
        const __nv_bfloat162 z = __hfma2(k2, hi2, __hmul2(k2, lo2));
        y[e] = *reinterpret_cast<const uint32_t*>(&z);
      }
      *reinterpret_cast<uint4*>(k_s + x * kLpBox + lp_swz(r, c)) =
          make_uint4(y[0], y[1], y[2], y[3]);
    }
  }
}

// 32 entries of row r of the transposed state (columns 32 j ..) as bf16 hi and
// lo tiles.
__device__ __forceinline__ void lp_store_state(uint8_t* hi_s, uint8_t* lo_s, int r, int j,
                                               const uint32_t (&x)[32]) {
  const unsigned long long neg1 = pk(-1.0f, -1.0f);
#pragma unroll
  for (int c = 0; c < 4; ++c) {
    uint32_t y[4], z[4];
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const float a = __uint_as_float(x[8 * c + 2 * e]), b = __uint_as_float(x[8 * c + 2 * e + 1]);
      y[e] = pack_bf16x2(a, b);
      const float2 rem = upk(fma2(pk(bf16_lo(y[e]), bf16_hi(y[e])), neg1, pk(a, b)));
      z[e] = pack_bf16x2(rem.x, rem.y);
    }
    const int off = (j >> 1) * kLpBox + lp_swz(r, 4 * (j & 1) + c);
    *reinterpret_cast<uint4*>(hi_s + off) = make_uint4(y[0], y[1], y[2], y[3]);
    *reinterpret_cast<uint4*>(lo_s + off) = make_uint4(z[0], z[1], z[2], z[3]);
  }
}

// Byte offset of column j of row i in a slot's tile as the TMA lays it out:
// [column / 64][D_k rows][64 columns], 128-byte swizzle.
template <int DK>
__device__ __forceinline__ int lp_tile_offset(int i, int j) {
  return (j >> 6) * DK * 128 + lp_swz(i, (j & 63) >> 3) + (j & 7) * 2;
}

// The address that `lane` gives to ldmatrix or stmatrix for piece j of a slot's
// tile: 16 columns (half j & 1 of warp wq's 32) by 16 rows (from 8 (j & ~1)), as
// four 8 x 8 matrices whose rows are the tile's: columns 0-7 and 8-15 of rows
// 0-7, then of rows 8-15.
template <int DK>
__device__ __forceinline__ int lp_piece_offset(int j, int wq, int lane) {
  return lp_tile_offset<DK>(8 * (j & ~1) + (lane & 7) + 8 * (lane >> 4),
                            32 * wq + 16 * (j & 1) + (lane & 8));
}

// A tile of a tensor map into L2 (the coordinates of the load that follows).
__device__ __forceinline__ void lp_prefetch_3d(const CUtensorMap* map, int x, int y, int z) {
  asm volatile("cp.async.bulk.prefetch.tensor.3d.L2.global.tile [%0, {%1, %2, %3}];" ::"l"(map),
               "r"(x), "r"(y), "r"(z)
               : "memory");
}

// Set `flag` behind this thread's view of memory; wait for it, bounded.
__device__ __forceinline__ void lp_set_flag(int* flag) {
  asm volatile("st.release.gpu.global.b32 [%0], %1;" ::"l"(flag), "r"(1) : "memory");
}
__device__ __forceinline__ bool lp_wait_flag(const int* flag) {
  const long long limit = abandonable_wait_limit();
  const long long t0 = clock64();
  for (;;) {
    int v;
    asm volatile("ld.acquire.gpu.global.b32 %0, [%1];" : "=r"(v) : "l"(flag) : "memory");
    if (v != 0) return true;
    if (clock64() - t0 > limit) return false;
    __nanosleep(64);
  }
}

template <int DK>
__global__ void __launch_bounds__(kLpThreads, 1)
    linear_prefill_kernel(const __grid_constant__ CUtensorMap q_map,
                          const __grid_constant__ CUtensorMap k_map,
                          const __grid_constant__ CUtensorMap v_map,
                          const __grid_constant__ CUtensorMap o_map,
                          const __grid_constant__ CUtensorMap pool_map,
                          const LinearPrefillParams prm) {
  using Shape = LpShape<DK>;
  constexpr int kBoxes = Shape::kBoxes, kStages = Shape::kStages;
  const LinearParams& p = prm.p;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;

  extern __shared__ __align__(16) uint8_t smem_raw[];
  const uint32_t raw = smem_addr(smem_raw);
  uint8_t* smem = smem_raw + (((raw + 1023u) & ~1023u) - raw);
  uint64_t* bars = reinterpret_cast<uint64_t*>(smem + Shape::kBarOff);
  float* diag = reinterpret_cast<float*>(smem + Shape::kPowOff);  // lambda^0 .. lambda^31
  LpWork* works = reinterpret_cast<LpWork*>(smem + Shape::kWorkOff);
  int* before = reinterpret_cast<int*>(smem + Shape::kLenOff);    // stream: see LpWalk
  const uint32_t bar0 = smem_addr(bars);
  const uint32_t q_full = bar0;                    // + 8 st: q landed
  const uint32_t k_full = bar0 + 8 * kStages;      // + 8 st: k landed
  const uint32_t v_full = bar0 + 16 * kStages;     // + 8 st: v landed
  const uint32_t q_free = bar0 + 24 * kStages;     // + 8 st: q read for the last time
  const uint32_t k_free = bar0 + 32 * kStages;     // + 8 st: k and the S_lo in its place read
  const uint32_t v_free = bar0 + 40 * kStages;     // + 8 st: the output has left the v stage
  const uint32_t bar1 = bar0 + 48 * kStages;
  const uint32_t p_raw = bar1, p_ready = bar1 + 8, k_ready = bar1 + 16, s_ready = bar1 + 24,
                 s_raw = bar1 + 32, o_raw = bar1 + 40, i_raw = bar1 + 48, i_ready = bar1 + 56,
                 drained = bar1 + 64, slot_full = bar1 + 72, slot_free = bar1 + 80;
  const uint32_t work_full = bar1 + 8 * kLpBars;     // + 8 e: entry e of the ring written
  const uint32_t work_free = work_full + 8 * kLpWorks;  // + 8 e: read by everyone
  uint32_t* tmem_slot =
      reinterpret_cast<uint32_t*>(bars + 6 * kStages + kLpBars + 2 * kLpWorks);
  volatile int* abort_word = reinterpret_cast<volatile int*>(tmem_slot + 1);

  // this CTA's stretches
  LpWalk walk{prm, before, static_cast<int>(blockIdx.x), 0, 0};
  if (prm.stream) {
    int L = 0;
    if (tid < p.B) {
      int s_, n_;
      linear_item(p, tid, s_, L, n_);
      before[tid + 1] = (L + kLpChunk - 1) / kLpChunk * (p.H_v * prm.slices / prm.team);
    }
    if (tid == 0) before[0] = 0;
    __syncthreads();
    if (warp == 0) {  // running sums, 32 items at a time
      int carry = 0;
      for (int i = 0; i < p.B; i += 32) {
        int x = i + lane < p.B ? before[i + lane + 1] : 0;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
          const int y = __shfl_up_sync(0xffffffffu, x, o);
          if (lane >= o) x += y;
        }
        if (i + lane < p.B) before[i + lane + 1] = carry + x;
        carry += __shfl_sync(0xffffffffu, x, 31);
      }
    }
    __syncthreads();
    walk.share(before[p.B], static_cast<int>(gridDim.x) / prm.team);
  } else {
    int s_, L, n_;
    linear_item(p, blockIdx.x / prm.segments / prm.slices / p.H_v, s_, L, n_);
    walk.segment(L);
  }
  LpWork w{};
  // The next stretch from the ring, for the lanes of a warp together; false at the
  // end, or when it did not come. A group of warps votes on it: one of them may
  // give up where the others were just let through.
  int n_works = 0;
  const auto next_work = [&]() {
    const int e = n_works % kLpWorks;
    bool ok =
        __all_sync(0xffffffffu, mbar_wait_abandonable(work_full + 8 * e, (n_works / kLpWorks) & 1,
                                                      abort_word, kErrConsumerWait));
    if (n_works == 1 && test_give_up(static_cast<int>(blockIdx.x), warp, 0)) {
      flag_error(kErrConsumerWait);
      *abort_word = 1;
      ok = false;
    }
    if (!ok) return false;
    w = works[e];
    __syncwarp();
    if (lane == 0) mbar_arrive(work_free + 8 * e);
    ++n_works;
    return w.n > 0;
  };

  // The loader, warp 0's first lane, starts on the first chunk ahead of the set-up
  // of the CTA (it waits for nobody); the rest follows below.
  const bool loads = !test_hold_tile(static_cast<int>(blockIdx.x));
  int issued[3] = {0, 0, 0};  // loads of q, k and v
  int slots = 0;              // and of slots
  const auto load = [&](int kind, const CUtensorMap* map, int c, int x0, int z, int boxes) {
    const int st = issued[kind] % kStages;
    const uint32_t bar = q_full + 8 * (kind * kStages + st);
    const uint32_t dst = smem_addr(smem + st * Shape::kStageBytes + kind * kBoxes * kLpBox);
    mbar_expect_tx(bar, boxes * kLpBox);
#pragma unroll 1
    for (int x = 0; x < boxes; ++x)
      tma_load_3d(dst + x * kLpBox, map, x0 + 64 * x, c * kLpChunk, z, bar);
    mbar_arrive(bar);
    ++issued[kind];
  };
  const auto load_slot = [&]() {  // where S_hi will be
    mbar_expect_tx(slot_full, w.cols / 64 * DK * 128);
#pragma unroll 1
    for (int x = 0; x < w.cols / 64; ++x)
      tma_load_3d(smem_addr(smem + Shape::kStateOff + x * DK * 128), &pool_map, w.col0 + 64 * x, 0,
                  w.slot_row, slot_full);
    mbar_arrive(slot_full);
    ++slots;
  };
  if (tid == 0) {
    for (int x = 0; x < 6 * kStages; ++x) mbar_init(bar0 + 8 * x, 1);
    mbar_init(p_raw, 1);
    mbar_init(p_ready, 128);
    mbar_init(k_ready, 128);
    mbar_init(s_ready, 128);
    mbar_init(s_raw, 1);
    mbar_init(o_raw, 1);
    mbar_init(i_raw, 1);
    mbar_init(i_ready, 128);
    mbar_init(drained, 1);
    mbar_init(slot_full, 1);
    mbar_init(slot_free, 1);
    for (int e = 0; e < kLpWorks; ++e) {
      mbar_init(work_full + 8 * e, 1);
      mbar_init(work_free + 8 * e, kLpReaders);
    }
    *abort_word = 0;
    fence_mbar_init();
    fence_async_smem();
    walk.next(w);
    works[0] = w;
    if (loads && w.n > 0) {
      load(0, &q_map, w.c0, 0, w.qk, kBoxes);
      load(1, &k_map, w.c0, 0, w.qk, kBoxes);
      if (w.whole_start) load_slot();
      load(2, &v_map, w.c0, w.col0, w.bh, w.cols / 64);
    }
    mbar_arrive(work_full);
  }
  __syncwarp();
  if (warp == 1) {
    tmem_alloc(smem_addr(tmem_slot), kLpTmemCols);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;

  // A role takes the stretches from the ring, and g counts the chunks of all of
  // them: the stages and the phases of the barriers go by it.
  if (warp < 4) lp_regs_dec<kLpRegsFew>();
  if (warp == 0) {
    // ------------------------------------------------------------ load
    bool ok = true;
    int g = 0;
    while (ok && next_work()) {
      if (lane == 0 && loads) {
        for (int i = 0; i < w.n; ++i, ++g) {
          if (g == 0) continue;  // on its way already
          const int st = g % kStages;
          const uint32_t use = (g / kStages) & 1;
          // S_lo of a chunk sits in the k stage of the chunk before it, the very
          // first in the last stage: that one is freed once before its first load
          const uint32_t k_phase = st == kStages - 1 ? use : use ^ 1;
          ok = mbar_wait_abandonable(q_free + 8 * st, use ^ 1, abort_word, kErrProducerWait);
          if (!ok) break;
          load(0, &q_map, w.c0 + i, 0, w.qk, kBoxes);
          // With two stages S_lo leaves k's place just before k is needed: into L2
          // with it meanwhile (2.49 us a chunk against 2.60). With three the place
          // is free long before, and the prefetch only costs (2.03 against 2.00).
          if (kStages == 2) {
#pragma unroll 1
            for (int x = 0; x < kBoxes; ++x)
              lp_prefetch_3d(&k_map, 64 * x, (w.c0 + i) * kLpChunk, w.qk);
          }
          ok = mbar_wait_abandonable(k_free + 8 * st, k_phase, abort_word, kErrProducerWait);
          if (!ok) break;
          load(1, &k_map, w.c0 + i, 0, w.qk, kBoxes);
          if (i == 0 && w.whole_start) {  // S_hi's place is free after the stretch before
            ok = mbar_wait_abandonable(slot_free, (slots & 1) ^ 1, abort_word, kErrProducerWait);
            if (!ok) break;
            load_slot();
          }
          ok = mbar_wait_abandonable(v_free + 8 * st, use ^ 1, abort_word, kErrProducerWait);
          if (!ok) break;
          load(2, &v_map, w.c0 + i, w.col0, w.bh, w.cols / 64);
        }
      }
      ok = __shfl_sync(0xffffffffu, ok, 0);
    }
    if (lane == 0) {
      // no copy may outlive the CTA: the last load of every stage has landed
      for (int x = 0; x < 3; ++x)
        for (int i = issued[x] > kStages ? issued[x] - kStages : 0; i < issued[x]; ++i)
          if (!mbar_wait_bounded(q_full + 8 * (x * kStages + i % kStages), (i / kStages) & 1))
            flag_error(kErrDrainWait);
      if (slots > 0 && !mbar_wait_bounded(slot_full, (slots - 1) & 1)) flag_error(kErrDrainWait);
    }
  } else if (warp == 1) {
    // ------------------------------------------------------------ mma
    // The warp stays together (descriptors and addresses are uniform), one lane issues.
    const bool leader = elect_one();
    {
      constexpr uint32_t id_qk = umma_idesc_bf16<128, 128, false, false>();
      constexpr uint32_t id_pv = umma_idesc_bf16<128, 128, false, true>();
      constexpr uint32_t id_kv = umma_idesc_bf16<128, DK, true, true>();
      const uint64_t s_desc =
          umma_desc(smem_addr(smem + Shape::kStateOff), 16, 1024, kUmmaSwizzle128);
      auto wait = [&](uint32_t bar, uint32_t phase) {
        const bool done = __all_sync(
            0xffffffffu, mbar_wait_abandonable(bar, phase, abort_word, kErrConsumerWait));
        tc_fence_after();
        return done;
      };
      bool ok = true;
      int g = 0;
      while (ok && next_work()) {
        for (int i = 0; i < w.n; ++i, ++g) {
          ok = false;  // until the end of the chunk
          const int st = g % kStages;
          const uint32_t ph = g & 1;
          const uint32_t q_s = smem_addr(smem + st * Shape::kStageBytes);
          const uint32_t k_s = q_s + kBoxes * kLpBox, v_s = k_s + kBoxes * kLpBox;
          const uint64_t q_k = umma_desc(q_s, 16, 1024, kUmmaSwizzle128);
          const uint64_t k_k = umma_desc(k_s, 16, 1024, kUmmaSwizzle128);
          const uint64_t k_mn = umma_desc(k_s, kLpBox, 1024, kUmmaSwizzle128);
          const uint64_t v_mn = umma_desc(v_s, kLpBox, 1024, kUmmaSwizzle128);
          const uint32_t use = (g / kStages) & 1;
          if (!wait(q_full + 8 * st, use) || !wait(k_full + 8 * st, use)) break;
          if (leader) {
#pragma unroll 2
            for (int ks = 0; ks < DK / 16; ++ks) {
              const uint32_t off = (ks >> 2) * kLpBox + (ks & 3) * 32;
              umma_bf16_at(tmem + kLpTmemP, q_k, off, k_k, off, id_qk, ks > 0);
            }
            umma_commit(p_raw);
          }
          __syncwarp();
          const bool from_slot = i == 0 && w.whole_start;
          if (!wait(from_slot ? slot_full : s_ready, from_slot ? slots & 1 : ph)) break;
          const int lo_st = (g + kStages - 1) % kStages;  // the k stage that holds S_lo
          if (from_slot) ++slots;
          if (leader) {
            if (from_slot) {
              // the slot's tile is S itself, rows of 64 columns: the other major-ness,
              // and bf16 has no S_lo
              const uint64_t tile_desc =
                  umma_desc(smem_addr(smem + Shape::kStateOff), DK * 128, 1024, kUmmaSwizzle128);
#pragma unroll 1
              for (int ks = 0; ks < DK / 16; ++ks)
                umma_bf16_at(tmem + kLpTmemInter, q_k, (ks >> 2) * kLpBox + (ks & 3) * 32,
                             tile_desc, ks * 2048, id_pv, ks > 0);
            } else {
              const uint64_t lo_desc =
                  umma_desc(smem_addr(smem + lo_st * Shape::kStageBytes + kBoxes * kLpBox), 16,
                            1024, kUmmaSwizzle128);
              // S_lo first: the next chunk's k waits for its place
#pragma unroll 1
              for (int half = 0; half < 2; ++half) {
                const uint64_t desc = half ? s_desc : lo_desc;
#pragma unroll 2
                for (int ks = 0; ks < DK / 16; ++ks) {
                  const uint32_t off = (ks >> 2) * kLpBox + (ks & 3) * 32;
                  umma_bf16_at(tmem + kLpTmemInter, q_k, off, desc, off, id_qk,
                               ks > 0 || half > 0);
                }
                if (half == 0) umma_commit(k_free + 8 * lo_st);
              }
            }
            umma_commit(i_raw);
            umma_commit(q_free + 8 * st);
          }
          __syncwarp();
          // A stretch that starts from its slot: the scaled slot is in TMEM, and the
          // state of the stretch before has left the k stage in which S_lo would be.
          if (from_slot && !wait(s_ready, ph)) break;
          if (from_slot && leader) umma_commit(k_free + 8 * lo_st);
          __syncwarp();
          if (!wait(v_full + 8 * st, use) || !wait(k_ready, ph)) break;
          if (leader) {
#pragma unroll 2
            for (int ks = 0; ks < kLpChunk / 16; ++ks)
              umma_bf16_at(tmem + kLpTmemState, v_mn, ks * 2048, k_mn, ks * 2048, id_kv, true);
            umma_commit(s_raw);
          }
          __syncwarp();
          // The first time round the instructions of P V are run once with the MMA
          // switched off, so that fetching them (3500 cycles, cold) falls into the wait.
          bool p_ok = true;
          for (int run = g > 0; run < 2; ++run) {
            if (run) p_ok = wait(p_ready, ph) && wait(i_ready, ph);
            if (!p_ok) break;
            if (leader) {
#pragma unroll 2
              for (int ks = 0; ks < kLpChunk / 16; ++ks)
                umma_bf16_ts_at(tmem + kLpTmemIntra, tmem + kLpTmemP + 8 * ks, v_mn, ks * 2048,
                                id_pv, true, run != 0);
            }
            __syncwarp();
          }
          if (!p_ok) break;
          if (leader) umma_commit(o_raw);
          __syncwarp();
          ok = true;
        }
      }
      if (leader) {
        umma_commit(drained);
        if (!mbar_wait_bounded(drained, 0)) flag_error(kErrDrainWait);
      }
    }
  } else if (warp == 2) {
    // ------------------------------------------------------------ walk
    if (lane == 0) {
      w = works[0];  // the first one comes from the loader
      walk.hi = w.rest;
      for (int k = 1; w.n > 0; ++k) {
        const int e = k % kLpWorks;
        if (!mbar_wait_abandonable(work_free + 8 * e, ((k / kLpWorks) & 1) ^ 1, abort_word,
                                   kErrProducerWait))
          break;
        walk.next(w);
        works[e] = w;
        mbar_arrive(work_full + 8 * e);
      }
    }
  } else if (warp == 3) {
    // ------------------------------------------------------------ padding
    // tokens behind an item's last chunk: +0.0. A tile's own CTA (segment), or
    // every grid's width of tiles.
    lp_grid_wait();
    const int tiles = p.B * p.H_v * prm.slices;
    const int step = prm.stream ? static_cast<int>(gridDim.x) : tiles;
    for (int tile = prm.stream ? blockIdx.x : blockIdx.x / prm.segments; tile < tiles;
         tile += step) {
      const int bh = tile / prm.slices, col0 = (tile - bh * prm.slices) * kLpCols;
      const int sh = p.D_v - col0 < kLpCols ? 3 : 4;  // 16-byte pieces of a row: 8 or 16
      int s_, L, n_;
      linear_item(p, bh / p.H_v, s_, L, n_);
      int64_t from = static_cast<int64_t>((L + kLpChunk - 1) / kLpChunk) * kLpChunk;
      int64_t to = p.T;
      if (!prm.stream) {
        const int64_t first =
            static_cast<int64_t>(blockIdx.x % prm.segments) * prm.seg_chunks * kLpChunk;
        const int64_t last = first + static_cast<int64_t>(prm.seg_chunks) * kLpChunk;
        from = from > first ? from : first;
        to = to < last ? to : last;
      }
      // a warp writes 512 bytes a store, four stores a turn
      const int rows = 32 >> sh;
      const size_t step_rows = static_cast<size_t>(rows) * p.D_v;
      int64_t i = from + (lane >> sh);
      uint16_t* at = p.out + (static_cast<size_t>(bh) * p.T + i) * p.D_v + col0 +
                     (lane & ((1 << sh) - 1)) * 8;
      for (; i + 3 * rows < to; i += 4 * rows, at += 4 * step_rows) {
#pragma unroll
        for (int e = 0; e < 4; ++e)
          *reinterpret_cast<uint4*>(at + e * step_rows) = make_uint4(0u, 0u, 0u, 0u);
      }
      for (; i < to; i += rows, at += step_rows)
        *reinterpret_cast<uint4*>(at) = make_uint4(0u, 0u, 0u, 0u);
    }
  } else if (warp < 8) {
    // ------------------------------------------------------------ P
    lp_regs_inc<kLpRegsMany>();
    const int wq = warp & 3, t = tid & 127;
    const uint32_t base = tmem + kLpTmemP + (static_cast<uint32_t>(32 * wq) << 16);
    bool ok = true;
    int g = 0;
    // behind the vote the weights of the stretch before are no longer read
    while (ok && named_barrier_and(1, 128, next_work())) {
      const float log_decay = w.log_decay;
      if (wq == 0) diag[lane] = decay_power(log_decay, lane);
      named_barrier(1, 128);
      unsigned long long w2[16];  // lambda^{31-e}
#pragma unroll
      for (int e = 0; e < 16; ++e) w2[e] = pk(diag[31 - 2 * e], diag[30 - 2 * e]);
      for (int i = 0; i < w.n; ++i, ++g) {
        ok = __all_sync(0xffffffffu,
                        mbar_wait_abandonable(p_raw, g & 1, abort_word, kErrConsumerWait));
        if (!ok) break;
        tc_fence_after();
#pragma unroll 1
        for (int j = 0; j < 4; ++j) {
          uint32_t y[16];
          if (j <= wq) {
            uint32_t x[32];
            tmem_ld32(base + 32 * j, x);
            const float a = decay_power(log_decay, j < wq ? t - 32 * j - 31 : 0);
            tmem_wait_ld();
            if (j < wq) {
              // all 32 columns are behind row t: lambda^{t-c} as
              // lambda^{t-32j-31} lambda^{31-e}, two packed products a pair
              const unsigned long long a2 = pk(a, a);
#pragma unroll
              for (int e = 0; e < 16; ++e) {
                const float2 f = upk(mul2(mul2(pk(__uint_as_float(x[2 * e]),
                                                  __uint_as_float(x[2 * e + 1])), a2), w2[e]));
                y[e] = pack_bf16x2(f.x, f.y);
              }
            } else {
              // the diagonal block: what is ahead of row t is set to 0
              const float* pt = diag + lane;
#pragma unroll
              for (int e = 0; e < 16; ++e)
                y[e] = pack_bf16x2(
                    2 * e <= lane ? __uint_as_float(x[2 * e]) * pt[-2 * e] : 0.0f,
                    2 * e + 1 <= lane ? __uint_as_float(x[2 * e + 1]) * pt[-2 * e - 1] : 0.0f);
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
      ok = named_barrier_and(1, 128, ok);
    }
  } else if (warp < 12) {
    // ------------------------------------------------------------ out
    lp_regs_inc<kLpRegsMany>();
    const int wq = warp & 3, t = tid & 127;
    const uint32_t lanes = tmem + (static_cast<uint32_t>(32 * wq) << 16);
    const unsigned long long scale2 = pk(p.scale, p.scale);
    const bool elected = t == 0;
    int leaving = -1;  // the v stage that an output is leaving
    bool ok = true;
    int g = 0;
    while (ok && named_barrier_and(2, 128, next_work())) {
      const float inter = decay_power(w.log_decay, t + 1);
      const unsigned long long inter2 = pk(inter, inter);
      for (int i = 0; i < w.n; ++i, ++g) {
        const int st = g % kStages;
        const uint32_t valid = t < w.L - i * kLpChunk ? 0xffffffffu : 0u;  // padding: +0.0
        uint8_t* o_s = smem + st * Shape::kStageBytes + 2 * kBoxes * kLpBox;
        // S^T q times lambda^{t+1} to where P V will be added to it
        ok = __all_sync(0xffffffffu,
                        mbar_wait_abandonable(i_raw, g & 1, abort_word, kErrConsumerWait));
        if (ok) {
          tc_fence_after();
#pragma unroll 1
          for (int j = 0; j < 4; ++j) {
            uint32_t x[32];
            tmem_ld32(lanes + kLpTmemInter + 32 * j, x);
            tmem_wait_ld();
#pragma unroll
            for (int e = 0; e < 32; e += 2) {
              const float2 f =
                  upk(mul2(pk(__uint_as_float(x[e]), __uint_as_float(x[e + 1])), inter2));
              x[e] = __float_as_uint(f.x);
              x[e + 1] = __float_as_uint(f.y);
            }
            tmem_st32(lanes + kLpTmemIntra + 32 * j, x);
          }
          tmem_wait_st();
          tc_fence_before();
          mbar_arrive(i_ready);
        }
        // the output before has left its v stage by now
        if (elected && leaving >= 0) {
          bulk_wait_read_all();
          mbar_arrive(v_free + 8 * leaving);
          leaving = -1;
        }
        ok = ok && mbar_wait_abandonable(o_raw, g & 1, abort_word, kErrConsumerWait);
        ok = __all_sync(0xffffffffu, ok);
        if (ok) {
          tc_fence_after();
#pragma unroll 1
          for (int j = 0; j < 4; ++j) {
            uint32_t x[32];
            tmem_ld32(lanes + kLpTmemIntra + 32 * j, x);
            tmem_wait_ld();
#pragma unroll
            for (int c = 0; c < 4; ++c) {
              uint32_t y[4];
#pragma unroll
              for (int e = 0; e < 4; ++e) {
                const int k = 8 * c + 2 * e;
                const float2 f =
                    upk(mul2(pk(__uint_as_float(x[k]), __uint_as_float(x[k + 1])), scale2));
                y[e] = pack_bf16x2(f.x, f.y) & valid;
              }
              *reinterpret_cast<uint4*>(o_s + (j >> 1) * kLpBox + lp_swz(t, 4 * (j & 1) + c)) =
                  make_uint4(y[0], y[1], y[2], y[3]);
            }
          }
          tc_fence_before();
        }
        fence_async_smem();
        ok = named_barrier_and(2, 128, ok);
        if (!ok) break;
        if (elected) {
          for (int x = 0; x < w.cols / 64; ++x)
            tma_store_3d(&o_map, w.col0 + 64 * x, (w.c0 + i) * kLpChunk, w.bh,
                         smem_addr(o_s + x * kLpBox));
          bulk_commit_group();
          leaving = st;
        }
      }
    }
    if (elected) bulk_wait_all();
  } else {
    // ------------------------------------------------------------ state
    lp_regs_inc<kLpRegsMany>();
    const int wq = warp & 3, r = tid & 127;  // r: column j of S, row of k and v
    const uint32_t lanes = tmem + kLpTmemState + (static_cast<uint32_t>(32 * wq) << 16);
    uint8_t* s_s = smem + Shape::kStateOff;
    const bool elected = r == 0;
    bool ok = true;
    // A state written for the next CTA and not passed on yet: that happens a chunk
    // or two later, when its writes are done and the fence need not wait for them
    // (5000 cycles); but before this CTA itself waits for another one's state.
    bool hands = false;
    // Every warp comes here once for a state, also one that gave up before (the
    // state then stays here): none is left alone at the barrier.
    const auto pass_on = [&](bool good) {
      __threadfence();
      if (named_barrier_and(3, 128, good) && elected) lp_set_flag(prm.flags + blockIdx.x);
      hands = false;
    };
    int g = 0;
    while (ok && named_barrier_and(3, 128, next_work())) {
      const float log_decay = w.log_decay;
      bool sums = true;  // segments: what this thread looked up of the sums behind its start
      // the first state, scaled, into TMEM for the first sum; one that comes from
      // another CTA as hi and lo for its first S^T q too (a slot's tile serves that
      // as it is)
      {
        if (hands && !w.whole_start) pass_on(true);
        const float decay = decay_power(log_decay, w.L < kLpChunk ? w.L : kLpChunk);
        const float* start = prm.starts + 4 * r +
                             static_cast<size_t>(prm.stream ? blockIdx.x - prm.team : blockIdx.x) * DK *
                                 kLpCols;
        uint8_t* lo_s = smem + (g + kStages - 1) % kStages * Shape::kStageBytes + kBoxes * kLpBox;
        if (w.whole_start) {
          ok = mbar_wait_abandonable(slot_full, slots & 1, abort_word, kErrConsumerWait);
          ++slots;
        } else if (!prm.stream) {
          lp_grid_wait();  // the scan's results
          for (int e = r; e < static_cast<int>(blockIdx.x) % prm.segments; e += 128)
            sums = sums && __ldcg(prm.flags + blockIdx.x - e) != 0;
        } else if (elected) {
          // S_lo goes to the k stage that the stretch before left its slot's tile in:
          // the vote below lets nobody write there until that store has read it
          bulk_wait_read_all();
          ok = lp_wait_flag(prm.flags + blockIdx.x - prm.team);
          if (!ok) {
            flag_error(kErrConsumerWait);
            *abort_word = 1;
          }
        }
        ok = named_barrier_and(3, 128, ok);
        if (!ok) break;
        if (w.whole_start) {
          // 16 columns x 16 rows at a time: transposed on the way from shared memory
#pragma unroll 1
          for (int j = 0; j < DK / 8; ++j) {
            uint32_t y[4], x[8];
            ldmatrix_x4_trans(smem_addr(s_s + lp_piece_offset<DK>(j, wq, lane)), y);
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              x[2 * e] = __float_as_uint(bf16_lo(y[e]) * decay);
              x[2 * e + 1] = __float_as_uint(bf16_hi(y[e]) * decay);
            }
            tmem_st_16x16(lanes + ((16u * (j & 1)) << 16) + 16 * (j >> 1), x);
          }
        } else {
#pragma unroll 1
          for (int j = 0; j < DK / 32; j += 2) {
            uint32_t x[2][32];  // two blocks' loads are in flight together
#pragma unroll
            for (int e = 0; e < 16; ++e) {
              const float4 f =
                  __ldcg(reinterpret_cast<const float4*>(start + (8 * j + e) * 4 * kLpCols));
              uint32_t* y = x[e >> 3] + 4 * (e & 7);
              y[0] = __float_as_uint(f.x);
              y[1] = __float_as_uint(f.y);
              y[2] = __float_as_uint(f.z);
              y[3] = __float_as_uint(f.w);
            }
#pragma unroll
            for (int y = 0; y < 2; ++y) {
              lp_store_state(s_s, lo_s, r, j + y, x[y]);
#pragma unroll
              for (int e = 0; e < 32; ++e)
                x[y][e] = __float_as_uint(__uint_as_float(x[y][e]) * decay);
              tmem_st32(lanes + 32 * (j + y), x[y]);
            }
          }
        }
        if (elected) bulk_wait_read_all();  // the state of the stretch before has left
        tmem_wait_st();
        fence_async_smem();
        tc_fence_before();
        mbar_arrive(s_ready);
      }
      for (int i = 0; i < w.n; ++i, ++g) {
        const int st = g % kStages;
        const uint32_t use = (g / kStages) & 1;
        const int left = w.L - i * kLpChunk;
        const int Lc = left < kLpChunk ? left : kLpChunk;
        uint8_t* k_s = smem + st * Shape::kStageBytes + kBoxes * kLpBox;
        const float weight = r < Lc ? decay_power(log_decay, Lc - 1 - r) : 0.0f;
        // q k^T has read k (and waited for it to land)
        ok = mbar_wait_abandonable(k_full + 8 * st, use, abort_word, kErrConsumerWait) &&
             mbar_wait_abandonable(p_raw, g & 1, abort_word, kErrConsumerWait);
        ok = __all_sync(0xffffffffu, ok);
        if (!ok) break;
        lp_weight_row<kBoxes>(k_s, r, weight);
        if (Lc < kLpChunk) {  // rows of k and v behind the last token: zeros
          ok = __all_sync(0xffffffffu, mbar_wait_abandonable(v_full + 8 * st, use, abort_word,
                                                             kErrConsumerWait));
          if (!ok) break;
          if (r >= Lc) {  // v lies behind k
#pragma unroll 1
            for (int c = 0; c < 8 * (kBoxes + 2); ++c)
              *reinterpret_cast<uint4*>(k_s + (c >> 3) * kLpBox + lp_swz(r, c & 7)) =
                  make_uint4(0u, 0u, 0u, 0u);
          }
        }
        fence_async_smem();
        mbar_arrive(k_ready);

        // the sum is done and has read this chunk's k: its stage takes S_lo
        ok = __all_sync(0xffffffffu,
                        mbar_wait_abandonable(s_raw, g & 1, abort_word, kErrConsumerWait));
        if (hands && i == 1 && test_give_up(static_cast<int>(blockIdx.x), warp, 1)) {
          flag_error(kErrConsumerWait);
          *abort_word = 1;
          ok = false;
        }
        if (!ok) break;
        tc_fence_after();
        if (i + 1 == w.n) {
          // every S^T q of the stretch has read S_hi: the next slot may land there
          if (elected) mbar_arrive(slot_free);
          ++g;
          break;
        }
        const int next_L = left - Lc < kLpChunk ? left - Lc : kLpChunk;
        const float decay = decay_power(log_decay, next_L);
        const unsigned long long decay2 = pk(decay, decay);
#pragma unroll 1
        for (int j = 0; j < DK / 32; ++j) {
          uint32_t x[32];
          tmem_ld32(lanes + 32 * j, x);
          tmem_wait_ld();
          lp_store_state(s_s, k_s, r, j, x);
#pragma unroll
          for (int e = 0; e < 32; e += 2) {
            const float2 f =
                upk(mul2(decay2, pk(__uint_as_float(x[e]), __uint_as_float(x[e + 1]))));
            x[e] = __float_as_uint(f.x);
            x[e + 1] = __float_as_uint(f.y);
          }
          tmem_st32(lanes + 32 * j, x);
        }
        tmem_wait_st();
        fence_async_smem();
        tc_fence_before();
        mbar_arrive(s_ready);
        if (hands && i > 0) pass_on(true);
      }
      if (hands) pass_on(ok);
      // The stretch's last state: rounded once to the slot, through a tile in the
      // last chunk's k stage (two-byte stores to the slot itself took 8000 cycles), or
      // as it is to the next CTA. With segments the next one has its state from the
      // scan.
      uint8_t* tile = smem + (g + kStages - 1) % kStages * Shape::kStageBytes + kBoxes * kLpBox;
      if (ok && (w.whole_end || prm.stream)) {
        float* hand = prm.starts + 4 * r + static_cast<size_t>(blockIdx.x) * DK * kLpCols;
        if (w.whole_end) {
#pragma unroll 1
          for (int j = 0; j < DK / 8; ++j) {
            uint32_t x[8], y[4];
            tmem_ld_16x16(lanes + ((16u * (j & 1)) << 16) + 16 * (j >> 1), x);
            tmem_wait_ld();
#pragma unroll
            for (int e = 0; e < 4; ++e)
              y[e] = pack_bf16x2(__uint_as_float(x[2 * e]), __uint_as_float(x[2 * e + 1]));
            stmatrix_x4_trans(smem_addr(tile + lp_piece_offset<DK>(j, wq, lane)), y);
          }
        } else {
#pragma unroll 1
          for (int j = 0; j < DK / 16; ++j) {
            uint32_t x[16];
            tmem_ld16(lanes + 16 * j, x);
            tmem_wait_ld();
#pragma unroll
            for (int e = 0; e < 4; ++e)
              __stcg(reinterpret_cast<float4*>(hand + (4 * j + e) * 4 * kLpCols),
                     make_float4(__uint_as_float(x[4 * e]), __uint_as_float(x[4 * e + 1]),
                                 __uint_as_float(x[4 * e + 2]), __uint_as_float(x[4 * e + 3])));
          }
        }
      }
      fence_async_smem();
      ok = named_barrier_and(3, 128, ok && sums);  // no slot from a sum that is not there
      hands = ok && prm.stream && !w.whole_end;
      if (ok && w.whole_end && elected) {
        for (int x = 0; x < w.cols / 64; ++x)
          tma_store_3d(&pool_map, w.col0 + 64 * x, 0, w.slot_row,
                       smem_addr(tile + x * DK * 128));
        bulk_commit_group();
      }
    }
    if (ok && hands) pass_on(true);
    if (elected) bulk_wait_all();
  }

  // every warp arrives here: free the tensor memory once no thread can touch it
  __syncwarp();
  tc_fence_before();
  __syncthreads();
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc(tmem, kLpTmemCols);
  }
}

// ---------------------------------------------------------------- segments

// First pass: the sum of a segment that another one follows, which is
// prm.seg_chunks whole chunks:  sum_j lambda^{end-1-j} k_j v_j^T  over its
// tokens j, into the next segment's entry of prm.starts (fp32, laid out as it says
// there). The weights reach from the segment's end, so the chunks' products add up
// in TMEM and nothing waits for the state. Chunks whose weights are 0 in fp32 are
// summed like the others, since 0 times an infinity or NaN is not 0 (leaving them out
// took 3 to 6 us off the long call above). Every block says in prm.flags whether its
// sum is there; without one the item's slot is not written. 64 KB a chunk at
// D_k = 128: HBM bounds it once the segments fill the SMs.
template <int DK>
struct LsShape {
  static constexpr int kBoxes = DK / 64;
  static constexpr int kStages = 3;
  static constexpr int kStageBytes = (kBoxes + 2) * kLpBox;  // k, v
  static constexpr int kBarOff = kStages * kStageBytes;
  static constexpr int kSmem = 1024 + kBarOff + 8 * (3 * kStages + 2) + 16;
};
constexpr int kLsThreads = 192;  // load, mma, and four warps that weight k and store

template <int DK>
__global__ void __launch_bounds__(kLsThreads, 1)
    linear_segment_kernel(const __grid_constant__ CUtensorMap k_map,
                          const __grid_constant__ CUtensorMap v_map,
                          const LinearPrefillParams prm) {
  using Shape = LsShape<DK>;
  constexpr int kBoxes = Shape::kBoxes, kStages = Shape::kStages;
  const LinearParams& p = prm.p;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int seg = blockIdx.x % (prm.segments - 1);
  const int tile = blockIdx.x / (prm.segments - 1);
  const int slice = tile % prm.slices;
  const int bh = tile / prm.slices;
  const int h = bh % p.H_v, b = bh / p.H_v;
  const int col0 = slice * kLpCols;
  const int cols = p.D_v - col0 < kLpCols ? p.D_v - col0 : kLpCols;
  int s, L, n;
  linear_item(p, b, s, L, n);
  lp_grid_launch_next();
  const int64_t end = static_cast<int64_t>(seg + 1) * prm.seg_chunks * kLpChunk;
  if (L <= end) return;  // the item's last segment, or behind it
  const float log_decay = p.log_decay[h];
  const int c0 = seg * prm.seg_chunks, n_chunks = prm.seg_chunks;

  extern __shared__ __align__(16) uint8_t smem_raw[];
  const uint32_t raw = smem_addr(smem_raw);
  uint8_t* smem = smem_raw + (((raw + 1023u) & ~1023u) - raw);
  uint64_t* bars = reinterpret_cast<uint64_t*>(smem + Shape::kBarOff);
  const uint32_t full = smem_addr(bars);          // + 8 st: k and v landed
  const uint32_t ready = full + 8 * kStages;      // + 8 st: k weighted
  const uint32_t free_ = full + 16 * kStages;     // + 8 st: the product has read them
  const uint32_t summed = full + 24 * kStages, drained = summed + 8;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(bars + 3 * kStages + 2);
  volatile int* abort_word = reinterpret_cast<volatile int*>(tmem_slot + 1);
  if (tid == 0) {
    for (int st = 0; st < kStages; ++st) {
      mbar_init(full + 8 * st, 1);
      mbar_init(ready + 8 * st, 128);
      mbar_init(free_ + 8 * st, 1);
    }
    mbar_init(summed, 1);
    mbar_init(drained, 1);
    *abort_word = 0;
    fence_mbar_init();
  }
  __syncwarp();
  if (warp == 4) {
    tmem_alloc(smem_addr(tmem_slot), 128);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;

  // the test hook counts these blocks on from the main kernel's
  const bool loads = !test_hold_tile(
      static_cast<int>(gridDim.x / (prm.segments - 1) * prm.segments + blockIdx.x));
  bool stored = true;
  if (warp == 4) {
    // ------------------------------------------------------------ load
    if (lane == 0 && loads) {
      const int zk = b * p.H_qk + h / p.group;
      int issued = 0;
      for (int i = 0; i < n_chunks; ++i) {
        const int st = i % kStages;
        const int y = (c0 + i) * kLpChunk;
        const uint32_t dst = smem_addr(smem + st * Shape::kStageBytes);
        if (!mbar_wait_abandonable(free_ + 8 * st, ((i / kStages) & 1) ^ 1, abort_word,
                                   kErrProducerWait))
          break;
        mbar_expect_tx(full + 8 * st, (kBoxes + cols / 64) * kLpBox);
#pragma unroll
        for (int x = 0; x < kBoxes; ++x)
          tma_load_3d(dst + x * kLpBox, &k_map, 64 * x, y, zk, full + 8 * st);
        for (int x = 0; x < cols / 64; ++x)
          tma_load_3d(dst + (kBoxes + x) * kLpBox, &v_map, col0 + 64 * x, y, bh, full + 8 * st);
        mbar_arrive(full + 8 * st);
        ++issued;
      }
      for (int i = issued > kStages ? issued - kStages : 0; i < issued; ++i)
        if (!mbar_wait_bounded(full + 8 * (i % kStages), (i / kStages) & 1))
          flag_error(kErrDrainWait);
    }
  } else if (warp == 5) {
    // ------------------------------------------------------------ mma
    if (lane == 0) {
      constexpr uint32_t id_kv = umma_idesc_bf16<128, DK, true, true>();
      bool ok = true;
      for (int i = 0; i < n_chunks && ok; ++i) {
        const int st = i % kStages;
        const uint32_t k_s = smem_addr(smem + st * Shape::kStageBytes);
        const uint64_t k_mn = umma_desc(k_s, kLpBox, 1024, kUmmaSwizzle128);
        const uint64_t v_mn = umma_desc(k_s + kBoxes * kLpBox, kLpBox, 1024, kUmmaSwizzle128);
        ok = mbar_wait_abandonable(full + 8 * st, (i / kStages) & 1, abort_word,
                                   kErrConsumerWait) &&
             mbar_wait_abandonable(ready + 8 * st, (i / kStages) & 1, abort_word,
                                   kErrConsumerWait);
        if (!ok) break;
        tc_fence_after();
#pragma unroll
        for (int ks = 0; ks < kLpChunk / 16; ++ks)
          umma_bf16_at(tmem, v_mn, ks * 2048, k_mn, ks * 2048, id_kv, i > 0 || ks > 0);
        umma_commit(free_ + 8 * st);
      }
      if (ok) umma_commit(summed);
      umma_commit(drained);
      if (!mbar_wait_bounded(drained, 0)) flag_error(kErrDrainWait);
    }
  } else {
    // ------------------------------------------------------------ weights, store
    const int r = tid;
    bool ok = true;
    for (int i = 0; i < n_chunks; ++i) {
      const int st = i % kStages;
      const float weight = decay_power(log_decay, (n_chunks - i) * kLpChunk - 1 - r);
      ok = mbar_wait_abandonable(full + 8 * st, (i / kStages) & 1, abort_word, kErrConsumerWait);
      if (!__all_sync(0xffffffffu, ok)) break;
      lp_weight_row<kBoxes>(smem + st * Shape::kStageBytes, r, weight);
      fence_async_smem();
      mbar_arrive(ready + 8 * st);
    }
    ok = ok && mbar_wait_abandonable(summed, 0, abort_word, kErrConsumerWait);
    stored = __all_sync(0xffffffffu, ok);
    if (stored) {
      tc_fence_after();
      const uint32_t lanes = tmem + (static_cast<uint32_t>(32 * warp) << 16);
      float* dst = prm.starts +
                   (static_cast<size_t>(tile) * prm.segments + seg + 1) * DK * kLpCols + 4 * r;
#pragma unroll 1
      for (int j = 0; j < DK / 32; ++j) {
        uint32_t x[32];
        tmem_ld32(lanes + 32 * j, x);
        tmem_wait_ld();
#pragma unroll
        for (int e = 0; e < 8; ++e)
          *reinterpret_cast<float4*>(dst + (8 * j + e) * 4 * kLpCols) =
              make_float4(__uint_as_float(x[4 * e]), __uint_as_float(x[4 * e + 1]),
                          __uint_as_float(x[4 * e + 2]), __uint_as_float(x[4 * e + 3]));
      }
    }
  }

  __syncwarp();
  tc_fence_before();
  stored = __syncthreads_and(stored);
  if (tid == 0) prm.flags[static_cast<size_t>(tile) * prm.segments + seg + 1] = stored;
  if (warp == 4) {
    tc_fence_after();
    tmem_dealloc(tmem, 128);
  }
}

// The scan: entry g of prm.starts from the sum of segment g - 1 to the first
// state of segment g,  start_g = lambda^{segment} start_{g-1} + sum_{g-1}, and
// entry 0 to start_0, the slot. A thread takes one state value of one tile.
constexpr int kLscanThreads = 256;
template <int DK>
__global__ void __launch_bounds__(kLscanThreads) linear_scan_kernel(const LinearPrefillParams prm) {
  constexpr int kBlocks = DK * kLpCols / kLscanThreads;  // of a tile
  const LinearParams& p = prm.p;
  const int tile = blockIdx.x / kBlocks;
  const int e = (blockIdx.x % kBlocks) * kLscanThreads + threadIdx.x;
  const int row = e / (4 * kLpCols) * 4 + e % 4;
  const int col = (tile % prm.slices) * kLpCols + e / 4 % kLpCols;
  const int bh = tile / prm.slices;
  const int h = bh % p.H_v, b = bh / p.H_v;
  int s, L, n;
  linear_item(p, b, s, L, n);
  lp_grid_launch_next();
  const int tokens = prm.seg_chunks * kLpChunk;
  const int count = (L + tokens - 1) / tokens;  // segments of this item
  lp_grid_wait();  // the segments' sums (and, through this launch, for the next one too)
  if (count <= 1) return;
  const float decay = decay_power(p.log_decay[h], tokens);
  float* at = prm.starts + static_cast<size_t>(tile) * prm.segments * DK * kLpCols + e;
  float x = 0.0f;
  if (col < p.D_v)
    x = bf16_bits_to_f32(
        p.state_pool[((static_cast<size_t>(s) * p.H_v + h) * DK + row) * p.D_v + col]);
  *at = x;
#pragma unroll 4
  for (int g = 1; g < count; ++g) {
    float* here = at + static_cast<size_t>(g) * DK * kLpCols;
    x = fmaf(decay, x, *here);
    *here = x;
  }
}

}  // namespace gdr
