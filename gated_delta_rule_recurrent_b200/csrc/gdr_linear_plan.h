// The host's plan of a linear-attention prefill: which of the kernel's modes a
// call runs in, and the workspace it needs. A function of sizes alone, apart from
// the entry points so that it can be checked without a GPU.
#pragma once

#include <cstdint>

#include "gdr.h"
#include "gdr_linear_prefill.cuh"

namespace gdr {

// How a call's chunks are spread over the SMs.
//   more tiles than SMs: each SM takes an equal share of all chunks (`stream`), in
//     teams of tiles that read the same q and k;
//   fewer tiles and long prompts: each tile is cut into `segments`;
//   else: a CTA for each tile.
// Cutting costs a pass over k and v and two more launches. The rule is a fit at
// D_k = 128 (c chunks in n segments: about 23 + 3.8 c / n us against 12 + 2.5 c) and
// serves D_k = 64 too. Cut against whole, cold caches, us, around its border:
//   tiles x chunks   72 x 16  72 x 24  72 x 32  48 x 12  36 x 8  36 x 12  4 x 6  4 x 64
//   n                2        2        2        3        4       4        3      32
//   D_k = 128, cut   60       75       89       42       34      38       26     32
//              whole 53       72       90       41       31      41       25     158
//   D_k = 64, cut    46       58       71       34       28      32       20     28
//             whole  45       60       77       35       27      35       23     135
//   cut?             no       yes      yes      yes      yes     yes      no     yes
// so that near the border the wrong side costs up to a tenth, and far from it none is
// taken.
struct PrefillPlan {
  int slices = 1, segments = 1, seg_chunks = 1, team = 1, grid = 1;
  bool stream = false;
  int64_t states = 0;     // bytes of states in the workspace
  int64_t workspace = 0;  // and of all of it
};
inline PrefillPlan plan_prefill(const gdr_dims* d, int sms) {
  PrefillPlan s;
  if (d->T <= kMaxT) return s;  // the decode kernel's
  s.slices = (d->D_v + kLpCols - 1) / kLpCols;
  const int chunks = (d->T - 1) / kLpChunk + 1;
  s.seg_chunks = chunks;
  const long long tiles = static_cast<long long>(d->B) * d->H_v * s.slices;
  const int64_t state = static_cast<int64_t>(d->D_k) * kLpCols * 4;
  s.grid = static_cast<int>(tiles);
  if (tiles > sms && d->B <= kLpItems && tiles * chunks < 0x7fffffffLL) {
    s.stream = true;
    // tiles that read the same q and k run side by side, up to 8 of them, as long
    // as teams of that many leave no more than 1 in 16 SMs idle
    const int sharing = d->H_v / d->H_qk * s.slices;
    for (int m = 2; m <= 8; ++m)
      if (sharing % m == 0 && 16 * (sms % m) <= sms) s.team = m;
    s.grid = sms / s.team * s.team;
    s.states = s.grid * state;
    s.workspace = s.states + s.grid * 4;
    return s;
  }
  long long n = sms / tiles;
  if (n > chunks / 2) n = chunks / 2;
  if (n >= 2 && chunks * (25 * n - 38) > 110 * n) {
    s.seg_chunks = static_cast<int>((chunks - 1) / n + 1);
    s.segments = (chunks - 1) / s.seg_chunks + 1;
    s.grid = static_cast<int>(tiles) * s.segments;
    s.states = s.grid * state;
    s.workspace = s.states + s.grid * 4;
  }
  return s;
}

}  // namespace gdr
