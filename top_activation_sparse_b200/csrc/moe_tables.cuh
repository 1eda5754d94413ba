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

}  // namespace qs
