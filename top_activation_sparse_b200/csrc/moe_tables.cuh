// The routing of a mixture-of-experts call, from the workspace into shared
// memory, for the kernels that run after the routing one.
#pragma once

#include "moe.cuh"

namespace qs {

struct MoeTables {
  int16_t expert[kMoeMaxE], first[kMoeMaxE], count[kMoeMaxE];
  int32_t cum[kMoeMaxE + 1];                    // passes before each active expert
  int16_t token[kMoeMaxSlots];
  int active;
};

// by all threads of the block, after the wait for the kernel that routes; a
// barrier follows before the first use.  pass: tokens per pass
__device__ __forceinline__ void load_tables(const MoeArgs& a, MoeTables& t, int pass, int threads) {
  const int tid = threadIdx.x, A = min(__ldcg(a.table), kMoeMaxE);
  for (int i = tid; i < A; i += threads) {
    t.expert[i] = (int16_t)__ldcg(a.table + kMtExpert + i);
    t.first[i] = (int16_t)__ldcg(a.table + kMtFirst + i);
    t.count[i] = (int16_t)__ldcg(a.table + kMtCount + i);
  }
  for (int i = tid; i < a.T * a.top_k; i += threads) t.token[i] = (int16_t)__ldcg(a.table + kMtToken + i);
  if (tid == 0) t.active = A;
  __syncthreads();
  for (int i = tid; i <= A; i += threads) {
    int n = 0;
#pragma unroll 4
    for (int k = 0; k < i; ++k) n += (t.count[k] + pass - 1) / pass;
    t.cum[i] = n;
  }
}

// The down projection's items: (expert, range of neurons, tile of columns).  Ranges: S
// per pass over an expert's weights, about one item per CTA in all; the buffers hold
// max_splits.  (cum: by passes of kMoeDownTokens.)
struct MoeDownItem {
  int e, s, j0, j1, c0, cw, slot0, cnt, steps;   // columns [c0, c0 + cw), neurons [j0, j1)
};
__device__ __forceinline__ int moe_splits(const MoeArgs& a, const MoeTables& t) {
  return max(1, a.plan.grid / (t.cum[t.active] * a.plan.col_tiles));
}
__device__ __forceinline__ int moe_expert_splits(const MoeArgs& a, const MoeTables& t, int ai, int S) {
  return min(S * (t.cum[ai + 1] - t.cum[ai]), a.plan.max_splits);
}
__device__ __forceinline__ int moe_split_sum(const MoeArgs& a, const MoeTables& t, int S) {
  int n = 0;
  for (int ai = 0; ai < t.active; ++ai) n += moe_expert_splits(a, t, ai, S);
  return n;
}
// (whole steps of `step` neurons)
__device__ __forceinline__ MoeDownItem moe_down_item(const MoeArgs& a, const MoeTables& t, int item, int S, int cols, int step) {
  MoeDownItem d;
  int rest = item / a.plan.col_tiles, ai = 0, n = moe_expert_splits(a, t, 0, S);
  for (; rest >= n; n = moe_expert_splits(a, t, ++ai, S)) rest -= n;
  d.s = rest;
  d.e = t.expert[ai];
  const int all = (a.d_ff + step - 1) / step;
  const int s0 = (int)((long long)all * rest / n), s1 = (int)((long long)all * (rest + 1) / n);
  d.j0 = s0 * step;
  d.j1 = min(s1 * step, a.d_ff);
  d.steps = s1 - s0;
  d.c0 = item % a.plan.col_tiles * cols;
  d.cw = min(cols, a.d_model - d.c0);
  d.slot0 = t.first[ai];
  d.cnt = t.count[ai];
  return d;
}

}  // namespace qs
