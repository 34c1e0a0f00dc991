// Host-side print of how a linear-attention prefill spreads its chunks: the plan
// of a call, then one line for each stretch of each block, in the block's order.
// Built and run by tests/test_linear_schedule.py.
//   arguments: SMs, B, H_qk, H_v, D_k, D_v, T, pool, then B lengths and B slots
#include <cstdio>
#include <cstdlib>
#include <vector>

#include "gdr_linear_plan.h"

int main(int argc, char** argv) {
  std::vector<int> a;
  for (int i = 1; i < argc; ++i) a.push_back(std::atoi(argv[i]));
  if (a.size() < 8 || a.size() != 8 + 2 * static_cast<size_t>(a[1])) return 2;
  gdr_dims d{a[1], a[6], a[2], a[3], a[4], a[5], a[7], GDR_LAYOUT_KV};
  const gdr::PrefillPlan plan = gdr::plan_prefill(&d, a[0]);
  const std::vector<float> decay(d.H_v, -1.0f);
  gdr::LinearPrefillParams prm{};
  gdr::LinearParams& p = prm.p;
  p.log_decay = decay.data();
  p.seq_lengths = a.data() + 8;
  p.state_indices = a.data() + 8 + d.B;
  p.B = d.B;
  p.T = d.T;
  p.H_qk = d.H_qk;
  p.H_v = d.H_v;
  p.D_v = d.D_v;
  p.pool_size = d.pool_size;
  p.group = d.H_v / d.H_qk;
  prm.slices = plan.slices;
  prm.stream = plan.stream;
  prm.team = plan.team;
  prm.segments = plan.segments;
  prm.seg_chunks = plan.seg_chunks;
  std::printf("%d %d %d %d %d\n", static_cast<int>(plan.stream), plan.segments, plan.team,
              plan.grid, plan.seg_chunks);
  std::vector<int> before(d.B + 1);
  for (int b = 0; b < d.B; ++b) {
    int s, L, n;
    gdr::linear_item(p, b, s, L, n);
    before[b + 1] = before[b] + (L + gdr::kLpChunk - 1) / gdr::kLpChunk *
                                    (p.H_v * prm.slices / prm.team);
  }
  for (int block = 0; block < plan.grid; ++block) {
    gdr::LpWalk walk{prm, before.data(), block, 0, 0};
    if (plan.stream) {
      walk.share(before[p.B], plan.grid / plan.team);
    } else {
      int s, L, n;
      gdr::linear_item(p, block / plan.segments / plan.slices / p.H_v, s, L, n);
      walk.segment(L);
    }
    gdr::LpWork w{};
    for (walk.next(w); w.n > 0; walk.next(w))
      std::printf("%d %d %d %d %d %d %d %d %d\n", block, w.bh, w.col0, w.c0, w.n, w.L,
                  w.whole_start, w.whole_end, w.slot_row);
  }
  return 0;
}
