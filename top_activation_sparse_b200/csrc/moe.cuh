// Mixture-of-experts FFN layer for a few tokens (moe_kernel.cuh): arguments and plan.
#pragma once

#include "qs_internal.cuh"

namespace qs {

constexpr int kMoeMaxT = 64;          // tokens per launch
constexpr int kMoeMaxModel = QS_MOE_MAX_MODEL;
constexpr int kMoePartRows = 2048;    // rows of partial sums (splits x tokens x experts per token)

// counters, zero between calls
enum MoeCtl { MC_QUEUE = 0, MC_ROUTED = 1, MC_READY = 2, MC_HIDDEN = 3, MC_DOWN = 4, MC_EXIT = 5, MC_COUNT = 8 };

struct MoePlan {
  int grid = 0;
  int local = 0;            // every CTA evaluates the router for itself
  int one_token = 0;        // a CTA goes on from its neurons to their down rows
  int router_items = 0;     // queue items of the router
  int x_items = 0;          // ... of which look for x's powers (4-bit weights)
  int hidden_items = 0;     // ... of the hidden layer
  int out_items = 0;        // ... of the final sums
  int col_tiles = 0;        // column tiles of the down projection
  int tile_cols = 0;        // ... of this many columns
  int down_tokens = 0;      // tokens per pass of the down projection
  int down_pitch = 0, down_stages = 0;
  int hidden_tokens = 0;    // tokens per pass of the hidden layer
  int x_bytes = 0;          // shared memory of x (4-bit weights)
  int row_bytes = 0, scale_bytes = 0, stage_bytes = 0, pitch = 0, stage_rows = 0, stages = 0;   // the ring
  int max_splits = 0;       // splits of an expert's neurons the buffers hold
  int sum_steps = 0;        // 4-bit down projection: steps of 64 neurons per sum in tensor memory
  // four kernels (routing; h; the down projection; the sums) on the tensor cores
  // instead of one: moe_fp4_factors.cu and moe_fp4_down.cu, or moe_bf16_tensor.cu
  int tensor = 0;
};
MoePlan plan_moe_bf16(int T, int d_model, int d_ff, int n_experts, int top_k, bool y_bf16);
MoePlan plan_moe_fp4(int T, int d_model, int d_ff, int n_experts, int top_k, bool y_bf16);

struct MoeArgs {
  const __nv_bfloat16* x = nullptr;       // [T, d_model]
  int T = 0, d_model = 0, d_ff = 0, E = 0, top_k = 0;
  int drelu = 0;                          // else ReLU(u)^2 g
  int fp4 = 0;
  const __nv_bfloat16* router = nullptr;  // [E, d_model]
  // the matrix whose ReLU decides which neurons are open comes first: gate for
  // dReLU, up for squared ReLU.  [E, d_ff, d_model] bf16, or codes
  const uint8_t* w1 = nullptr;
  const uint8_t* w2 = nullptr;
  const uint8_t* wd = nullptr;
  const uint8_t* s1 = nullptr;            // MX scales [E, d_ff, d_model/32]
  const uint8_t* s2 = nullptr;
  const uint8_t* sd = nullptr;
  const float* b1 = nullptr;              // [E, d_ff] or NULL (dReLU)
  const float* b2 = nullptr;
  void* y = nullptr;                      // [T, d_model]
  int y_bf16 = 1;
  int32_t* experts = nullptr;             // [T, top_k] or NULL
  float* weights = nullptr;               // [T, top_k] or NULL
  // workspace
  int32_t* ctl = nullptr;                 // MC_COUNT counters
  float* logits = nullptr;                // [T, E]
  int32_t* table = nullptr;               // routing tables (see below)
  float* share = nullptr;                 // [T, top_k]
  float* xup = nullptr;                   // [T] power of two that takes x to float16 (4-bit weights)
  uint8_t* xt = nullptr;                  // [T, 8, d_model/2] x as eight 4-bit numbers (4-bit weights)
  uint8_t* xs = nullptr;                  // [T, moe_xs_pitch] scale bytes of the first of them
  float* h = nullptr;                     // [T * top_k, d_ff]; plan.tensor: [T * top_k, 3, d_ff] bf16
  uint8_t* nz = nullptr;                  // [min(E, T * top_k), d_ff]
  float* parts = nullptr;                 // [splits][T * top_k][d_model]
  DevStatus* status = nullptr;
  MoePlan plan{};
};
cudaError_t launch_moe_bf16(const MoeArgs& a, cudaStream_t s);
cudaError_t launch_moe_fp4(const MoeArgs& a, cudaStream_t s);
cudaError_t launch_moe_fp4_factors(const MoeArgs& a, cudaStream_t s);
cudaError_t launch_moe_fp4_down(const MoeArgs& a, cudaStream_t s);
cudaError_t launch_moe_bf16_tensor(const MoeArgs& a, cudaStream_t s);
cudaError_t launch_moe_sum(const MoeArgs& a, cudaStream_t s);
constexpr int kMoeDownTokens = 40;                        // tensor-core down projections: per pass
constexpr int kMoeDownCols = 512, kMoeDownColsBf16 = 256; // ... columns per item
__device__ __forceinline__ float relu_nan(float v) { return v <= 0.0f ? 0.0f : v; }   // keeps a NaN
constexpr int kMoeXTerms = 8;
__host__ __device__ constexpr int moe_xs_pitch(int d_model) { return (d_model / 32 + 31) / 32 * 32; }

// routing tables, int32: [0] active experts A, then per active expert its
// number, first slot and number of tokens, then per slot its token, then per
// (token, choice) its slot
constexpr int kMoeMaxE = 256, kMoeMaxK = 16, kMoeMaxSlots = kMoeMaxT * kMoeMaxK;
constexpr int kMtExpert = 8, kMtFirst = kMtExpert + kMoeMaxE, kMtCount = kMtFirst + kMoeMaxE,
              kMtToken = kMtCount + kMoeMaxE, kMtSlot = kMtToken + kMoeMaxSlots, kMtSize = kMtSlot + kMoeMaxSlots;

}  // namespace qs
