// A whole mixture-of-experts FFN layer in one kernel: one token, or several of large
// bf16 experts (make_plan says when).  Included by moe_bf16.cu and moe_fp4.cu, which say with
// what weights (kFp4).  (Everything else: the routing kernel below, then
// moe_bf16_tensor.cu, or moe_fp4_factors.cu and moe_fp4_down.cu.)
//
//   logits = x W_r^T;  each token's top_k largest (ties: lower expert) are its
//   experts, p = softmax over them;  for each (token, expert e):
//     h = ReLU(g + b_g) ReLU(u + b_u)   or   ReLU(u)^2 g,   g, u = x W_gate[e]^T, x W_up[e]^T
//   y = sum_e p_e h W_down[e]
//
// Bound by the bytes of the experts' weights.  All three matrices are stored
// neuron by neuron ([E, d_ff, d_model]): neuron j's gate, up and down weights
// are contiguous rows.  The factor whose ReLU can close a neuron is computed
// first, for every neuron; the other matrix's row is read only where some
// token's first factor is not 0, the down row only where some token's h is
// not 0 (exact: a closed neuron contributes 0).
//
// One launch, no grid barrier: CTAs draw items from one queue (an atomic
// counter), in four kinds, in this order:
//   router  logits of 16 experts x 8 tokens per item; the CTA that finishes the
//           last of them selects the experts and lists each expert's tokens;
//   hidden  an equal share of the active experts' neurons: first factor, then
//           the second for the open neurons, h, and a flag per neuron;
//   down    (expert, column strip, range of neurons): compacts its flagged
//           neurons, reads their down rows, leaves partial sums;
//   sum     y from the partial sums, in a fixed order.
// An item waits only for items of earlier kinds.  Those were drawn before it
// by CTAs that run, and none of them waits for a later one, so the queue
// drains whatever part of the grid is resident (two calls at once share the
// SMs), and no result depends on which CTA does what.  Waits are bounded.
//
// The hidden layer's rows come through a ring in shared memory, filled by one
// warp with a bulk copy per row (a row is contiguous: 8 KB of bf16 at d_model =
// 4096).  Loading them from the warps straight to registers, 64 or 128 bytes of
// each of 16 rows at a time, reached 1.4 to 3.3 TB/s: DRAM wants its pages read
// in one go.  The order of the rows hides the dependence on what is open: first
// factors of batch b + 1, then second factors of batch b, and, with one token,
// the down rows of batch b - 1.
//
// Products run on mma.sync m16n8k16 (16 tokens x 8 neurons; 16 columns x 8
// tokens in the down projection): with weights read once, a few tokens stay
// bound by bytes.  x stays on the SM: with bf16 weights in registers, each warp
// holding its part of d_model for all tokens of the pass, with 4-bit weights (whose
// expansion needs the registers) in shared memory.  The sum over k may be permuted
// freely as long as both operands agree; a lane's 16 bytes are its k values.  x and
// bf16 weights enter exactly; h enters as the sum of three bf16 numbers (relative
// error below 2^-24).  4-bit weights are expanded in registers, exactly.
//
// 1 token, 2 of 8 dReLU experts of 14336 x 4096: bf16 76 us (46 at the memory's rate),
// 4-bit 65 (12: bound by the expansion, 1.5 instructions per cycle, and by latencies:
// about 7 us of routing, 4 for the first rows, 8 for the last sums).  2 tokens, 8 experts of
// 11008 x 4096, bf16: 138 us.
#pragma once

#include "fp4.cuh"
#include "moe.cuh"

namespace qs {
namespace {

// Warps that compute.  bf16 rows: 8, with 168 registers, in which x and a strip of
// columns fit (16 warps with 96: 521 against 447 us for 8 tokens, 8 experts of
// 4096 x 11008; a spill goes to L2, the ring leaves no L1).  4-bit rows, whose
// expansion waits for results at every step: 16 (67 against 79 us for one token,
// 4096 x 14336).
constexpr int kMWarps = kFp4 ? 16 : 8;
constexpr int kMThreads = kMWarps * 32;
constexpr int kThreads = kMThreads + 32;   // and one that copies
constexpr int kMaxNg = 2;              // groups of 8 tokens per pass
constexpr int kBatch = 64;             // neurons per batch (32 with two groups of tokens)
constexpr int kListD = 8 * kMThreads;  // neurons per round of the down projection
constexpr int kRowsD = 128;            // flagged neurons whose h is staged at a time
constexpr int kHPitch = kRowsD + 16;   // bf16 entries per token (pitch = 32 bytes mod 128)
constexpr int kTail = (kFp4 ? 172 : 176) * 1024;      // x (4-bit weights), then the ring of rows
constexpr int kMaxStages = 8;

struct Smem {
  unsigned char tail[kTail];
  union {
    float red[kMWarps * kBatch * 8];             // the warps' sums
    struct {
      __nv_bfloat16 h[3][8 * kMaxNg * kHPitch];
      uint16_t list[kListD];
    } d;
    int sel[kMoeMaxSlots + kMoeMaxE];            // choices by expert, then tokens per expert
  };
  float first[2][kBatch * 8];                    // first factors of two batches
  int rows[2][kBatch];                           // their open neurons
  int nrows[2];
  int drows[2][kBatch];                          // one token: neurons with h != 0, and p h
  float dval[2][kBatch];
  int ndrows[2];
  float hval[kBatch];
  uint32_t mask[kBatch / 4];
  // this call's routing
  int16_t expert[kMoeMaxE], firsts[kMoeMaxE], count[kMoeMaxE];
  int16_t token[kMoeMaxSlots], slot[kMoeMaxSlots];
  int16_t cum[2][kMoeMaxE + 1];                  // passes before each active expert (hidden layer, down)
  uint8_t slot_expert[kMoeMaxSlots];             // the active expert of a slot
  float share[kMoeMaxSlots];
  float xup[kMoeMaxT];                           // 4-bit weights: the power of two x is multiplied with
  int active;
  int tok[8 * kMaxNg];                           // the pass's tokens (-1: none)
  int scan[kMWarps];
  int item, last, abort;
  uint64_t full[kMaxStages], empty[kMaxStages], dfull[kMaxStages], dempty[kMaxStages];
  // lists of rows: written for the copying warp, read by it (0, 1: open neurons;
  // 2, 3: down rows)
  uint64_t listed[4], taken[4];
};
static_assert(sizeof(Smem) <= 227 * 1024 - 1024, "shared memory");

// (by name, not by reference: functions of their own would reach a reference
// through generic addresses)
__device__ __forceinline__ Smem& smem() {
  extern __shared__ __align__(128) unsigned char smem_raw[];
  return *reinterpret_cast<Smem*>(smem_raw);
}

// the computing warps' barrier
__device__ __forceinline__ void csync() { asm volatile("bar.sync 1, %0;" ::"n"(kMThreads) : "memory"); }

__device__ __forceinline__ uint4 ld_x(const __nv_bfloat16* p) {
  uint4 r;
  asm volatile("ld.global.nc.v4.u32 {%0,%1,%2,%3}, [%4];" : "=r"(r.x), "=r"(r.y), "=r"(r.z), "=r"(r.w) : "l"(p));
  return r;
}

__device__ __forceinline__ void mma_bf16(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                         uint32_t b1) {
  asm(
      "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// ---- queue and waits ---------------------------------------------------------
__device__ __forceinline__ int ld_acquire(const int32_t* p) {
  int v;
  asm volatile("ld.acquire.gpu.global.s32 %0, [%1];" : "=r"(v) : "l"(p) : "memory");
  return v;
}

// thread 0 waits until *p >= n; the computing warps leave together
__device__ __forceinline__ bool wait_for(const int32_t* p, int n, DevStatus* st, uint32_t where, Smem& sm) {
  if (threadIdx.x == 0) {
    uint32_t i = 0;
    bool ok = true;
    while (ok && ld_acquire(p) < n) {
      if (++i >= kWaitLimit) {
        dev_fail(st, DEV_TIMEOUT, where, (uint32_t)n);
        ok = false;
      }
      __nanosleep(32);
    }
    __threadfence();
    sm.last = ok;
  }
  csync();
  return sm.last != 0;
}

// the computing warps' writes are visible before the count goes up; the count
// before, to all of them
__device__ __forceinline__ int finish(int32_t* p, Smem& sm) {
  __threadfence();
  csync();
  if (threadIdx.x == 0) sm.last = atomicAdd(p, 1);
  csync();
  return sm.last;
}

// bounded wait on a barrier of this CTA; after one that gave up, none waits
__device__ __forceinline__ bool ring_wait(uint64_t* b, uint32_t parity, Smem& sm, DevStatus* st, uint32_t where) {
  for (uint32_t i = 0; i < kWaitLimit; ++i) {
    if (mbar_try_wait(b, parity)) return true;
    if ((i & 15u) == 15u && *(volatile int*)&sm.abort) return false;
  }
  dev_fail(st, DEV_TIMEOUT, where, 0u);
  atomicExch(&sm.abort, 1);
  return false;
}

// ---- router ------------------------------------------------------------------
// Partial logits of 16 experts x 8 tokens (16 x 8 matrix instructions; the warps
// share d_model) to part[expert * 8 + token] of each warp.
__device__ __forceinline__ void router_tile(const MoeArgs& a, int e0, int t0, float* part, int lane, int warp) {
  const int g = lane >> 2, q = lane & 3, units = a.d_model / 32;
  const bool ok0 = e0 + g < a.E, ok1 = e0 + 8 + g < a.E, okx = t0 + g < a.T;
  const __nv_bfloat16* w0 = a.router + (size_t)(ok0 ? e0 + g : 0) * a.d_model + q * 8;
  const __nv_bfloat16* w1 = a.router + (size_t)(ok1 ? e0 + 8 + g : 0) * a.d_model + q * 8;
  const __nv_bfloat16* x = a.x + (size_t)(okx ? t0 + g : 0) * a.d_model + q * 8;
  float acc[2][4] = {{0.0f, 0.0f, 0.0f, 0.0f}, {0.0f, 0.0f, 0.0f, 0.0f}};
  const uint4 z = make_uint4(0, 0, 0, 0);
#pragma unroll 8
  for (int u = warp; u < units; u += kMWarps) {
    const uint4 v0 = ok0 ? ld_x(w0 + u * 32) : z, v1 = ok1 ? ld_x(w1 + u * 32) : z, b = okx ? ld_x(x + u * 32) : z;
    mma_bf16(acc[0], v0.x, v1.x, v0.y, v1.y, b.x, b.y);
    mma_bf16(acc[1], v0.z, v1.z, v0.w, v1.w, b.z, b.w);
  }
  float* o = part + g * 8 + 2 * q;
  *reinterpret_cast<float2*>(o) = make_float2(acc[0][0] + acc[1][0], acc[0][1] + acc[1][1]);
  *reinterpret_cast<float2*>(o + 64) = make_float2(acc[0][2] + acc[1][2], acc[0][3] + acc[1][3]);
}

// item: one such tile, to the workspace
__device__ __noinline__ void router_item(const MoeArgs& a, int item, int lane, int warp) {
  Smem& sm = smem();
  const int groups = (a.T + 7) / 8, e0 = item / groups * 16, t0 = item % groups * 8;
  router_tile(a, e0, t0, sm.red + warp * 128, lane, warp);
  csync();
  const int e = e0 + (threadIdx.x >> 3), t = t0 + (threadIdx.x & 7);
  if (threadIdx.x < 128 && e < a.E && t < a.T) {
    float v = 0.0f;
#pragma unroll
    for (int w = 0; w < kMWarps; ++w) v += sm.red[w * 128 + threadIdx.x];
    __stcg(a.logits + (size_t)t * a.E + e, v);
  }
}

// The power of two that brings a token's largest |x| into [2^14, 2^15).
__device__ __forceinline__ float x_power(const __nv_bfloat16* x, int d, int lane) {
  uint32_t m = 0;
#pragma unroll 4
  for (int k = lane * 8; k < d; k += 256) {
    const uint4 v = ld_x(x + k);
    const uint32_t u[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) m = max(m, max(u[i] & 0x7fffu, (u[i] >> 16) & 0x7fffu));
  }
#pragma unroll
  for (int i = 16; i; i >>= 1) m = max(m, __shfl_xor_sync(0xffffffffu, m, i));
  const int e = (int)(m >> 7);                      // biased exponent of the largest
  // (nothing but subnormal numbers, or a non-finite one: no useful power);
  // at most 2^126, so that its reciprocal is a normal number
  const int up = e == 0 || e == 255 ? 0 : min(126, 127 + 14 - e);
  return __uint_as_float((uint32_t)(up + 127) << 23);
}

// larger float, larger key (NaN above all), and back
__device__ __forceinline__ uint32_t order_key(float f) {
  if (f != f) return 0xffffffffu;
  const uint32_t u = __float_as_uint(f == 0.0f ? 0.0f : f);
  return (u & 0x80000000u) ? ~u : (u | 0x80000000u);
}
__device__ __forceinline__ float key_value(uint32_t k) {
  return __uint_as_float((k & 0x80000000u) ? k ^ 0x80000000u : ~k);
}

// Experts and shares of every token from logits [T, E], then the experts' token
// lists, into sm.  (logits may be the union's memory: they are read before a
// barrier, the choices are written to it after.)  Run once per call, by cold
// code, whose instructions come from L2: short loops, not unrolled ones (32 tokens, 2
// of 8 experts: 26 K -> 7 K cycles).
template <bool SHARED>
__device__ __noinline__ void select_experts(const MoeArgs& a, const float* logits, bool publish, int lane, int warp) {
  Smem& sm = smem();
  const int K = a.top_k, n = a.T * K;
#pragma unroll 1
  for (int t = warp; t < a.T; t += kMWarps) {
    uint32_t taken = 0;                       // bit i: this lane's expert lane + 32 i is chosen
    float best = 0.0f, sum = 0.0f, mine = 0.0f;
    int choice = 0;                           // lane j: choice j
#pragma unroll 1
    for (int j = 0; j < K; ++j) {
      uint32_t key = 0;                       // (a real key is never 0)
      int at = kMoeMaxE;
#pragma unroll 1
      for (int e = lane; e < a.E; e += 32) {
        const uint32_t k = order_key(SHARED ? logits[t * a.E + e] : __ldcg(logits + (size_t)t * a.E + e));
        if (k > key && !((taken >> (e >> 5)) & 1u)) key = k, at = e;
      }
      const uint32_t top = __reduce_max_sync(0xffffffffu, key);
      const int e = __reduce_min_sync(0xffffffffu, key == top ? at : kMoeMaxE);
      if (at == e) taken |= 1u << (e >> 5);
      const float l = key_value(top);
      if (j == 0) best = l;
      const float p = expf(l - best);
      sum += p;
      if (lane == j) mine = p, choice = e;
    }
    if (lane < K) {
      const float p = mine / sum;
      sm.slot[t * K + lane] = (int16_t)choice;     // the expert, for now
      sm.share[t * K + lane] = p;
      if (publish) {
        if (a.experts) a.experts[t * K + lane] = choice;
        if (a.weights) a.weights[t * K + lane] = p;
      }
    }
  }
  csync();
  int* cnt = sm.sel + kMoeMaxSlots;
  for (int i = threadIdx.x; i < a.E; i += kMThreads) cnt[i] = 0;
  csync();
#pragma unroll 1
  for (int i = threadIdx.x; i < n; i += kMThreads) {
    sm.sel[i] = sm.slot[i];
    atomicAdd(&cnt[sm.slot[i]], 1);
  }
  csync();
  // experts without tokens drop out: sums over the experts before of (active
  // experts, slots), both below 2^16
  const int e = threadIdx.x, c = e < a.E ? cnt[e] : 0, v = ((c > 0) << 16) | c;
  int inc = v;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int u = __shfl_up_sync(0xffffffffu, inc, o);
    if (lane >= o) inc += u;
  }
  if (lane == 31) sm.scan[warp] = inc;
  csync();
  int before = 0, total = 0;
#pragma unroll
  for (int w = 0; w < kMWarps; ++w) {
    const int s = sm.scan[w];
    if (w < warp) before += s;
    total += s;
  }
  const int ex = before + inc - v;
  if (c > 0) {
    const int ai = ex >> 16;
    sm.expert[ai] = (int16_t)e;
    sm.firsts[ai] = (int16_t)(ex & 0xffff);
    sm.count[ai] = (int16_t)c;
  }
  if (threadIdx.x == 0) sm.active = total >> 16;
  csync();
  // a warp per active expert: its tokens in order
#pragma unroll 1
  for (int ai = warp; ai < sm.active; ai += kMWarps) {
    int at = sm.firsts[ai];
    const int ee = sm.expert[ai];
#pragma unroll 1
    for (int i0 = 0; i0 < n; i0 += 32) {
      const bool is = i0 + lane < n && sm.sel[i0 + lane] == ee;
      const unsigned m = __ballot_sync(0xffffffffu, is);
      if (is) {
        const int to = at + __popc(m & lanemask_lt());
        sm.token[to] = (int16_t)((i0 + lane) / K);
        sm.slot_expert[to] = (uint8_t)ai;
        sm.slot[i0 + lane] = (int16_t)to;
      }
      at += __popc(m);
    }
  }
  csync();
}

// passes over an expert's weights: what its neurons weigh when work is dealt out
__device__ __forceinline__ int passes_of(const Smem& sm, int kind, int ai) { return sm.cum[kind][ai + 1] - sm.cum[kind][ai]; }
__device__ __forceinline__ void count_passes(const MoeArgs& a, Smem& sm) {
  for (int i = threadIdx.x; i < 2 * (sm.active + 1); i += kMThreads) {
    const int kind = i & 1, ai = i >> 1, tokens = kind ? a.plan.down_tokens : a.plan.hidden_tokens;
    int n = 0;
#pragma unroll 4
    for (int k = 0; k < ai; ++k) n += (sm.count[k] + tokens - 1) / tokens;
    sm.cum[kind][ai] = (int16_t)n;
  }
}

// the routing from sm to the workspace, and back in every other CTA
__device__ void publish_routing(const MoeArgs& a, Smem& sm) {
  const int n = a.T * a.top_k, tid = threadIdx.x;
  for (int i = tid; i < sm.active; i += kMThreads) {
    __stcg(a.table + kMtExpert + i, (int)sm.expert[i]);
    __stcg(a.table + kMtFirst + i, (int)sm.firsts[i]);
    __stcg(a.table + kMtCount + i, (int)sm.count[i]);
  }
  for (int i = tid; i < n; i += kMThreads) {
    __stcg(a.table + kMtToken + i, (int)sm.token[i]);
    __stcg(a.table + kMtSlot + i, (int)sm.slot[i]);
    __stcg(a.share + i, sm.share[i]);
  }
  if (tid == 0) __stcg(a.table, sm.active);
}
__device__ void fetch_routing(const MoeArgs& a, Smem& sm) {
  const int n = a.T * a.top_k, tid = threadIdx.x, A = __ldcg(a.table);
  for (int i = tid; i < A; i += kMThreads) {
    sm.expert[i] = (int16_t)__ldcg(a.table + kMtExpert + i);
    sm.firsts[i] = (int16_t)__ldcg(a.table + kMtFirst + i);
    sm.count[i] = (int16_t)__ldcg(a.table + kMtCount + i);
  }
  for (int i = tid; i < n; i += kMThreads) {
    sm.token[i] = (int16_t)__ldcg(a.table + kMtToken + i);
    sm.slot[i] = (int16_t)__ldcg(a.table + kMtSlot + i);
    sm.share[i] = __ldcg(a.share + i);
  }
  if (a.fp4)
    for (int i = tid; i < a.T; i += kMThreads) sm.xup[i] = __ldcg(a.xup + i);
  if (tid == 0) sm.active = A;
  csync();
  for (int i = tid; i < n; i += kMThreads) {
    int ai = 0;
#pragma unroll 1
    for (int step = kMoeMaxE / 2; step; step >>= 1)
      if (ai + step < A && sm.firsts[ai + step] <= i) ai += step;
    sm.slot_expert[i] = (uint8_t)ai;
  }
}

// Local routing: at most 8 tokens and a small router (at most 64 experts and 128
// KB, from L2), which every CTA evaluates for itself: less time than handing
// the result over.  The warps share d_model; 16 experts x 8 tokens per matrix
// instruction.
__device__ __noinline__ void route_here(const MoeArgs& a, bool publish, int lane, int warp) {
  Smem& sm = smem();
  const int pairs = a.E * a.T;
  float* part = sm.red;                             // [warp][expert][8 tokens]: 64 x 8 x 8 at most
#pragma unroll 1
  for (int e0 = 0; e0 < a.E; e0 += 16) router_tile(a, e0, 0, part + warp * 512 + e0 * 8, lane, warp);
  if (a.fp4)
    for (int t = warp; t < a.T; t += kMWarps) {
      const float u = x_power(a.x + (size_t)t * a.d_model, a.d_model, lane);
      if (lane == 0) sm.xup[t] = u;
    }
  csync();
  float v[2] = {0.0f, 0.0f};                        // pairs <= 512
#pragma unroll
  for (int k = 0; k < 2; ++k) {
    const int i = threadIdx.x + k * kMThreads;      // token i / E, expert i % E
    if (i < pairs)
#pragma unroll
      for (int w = 0; w < kMWarps; ++w) v[k] += part[w * 512 + (i % a.E) * 8 + i / a.E];
  }
  csync();
#pragma unroll
  for (int k = 0; k < 2; ++k)
    if ((int)threadIdx.x + k * kMThreads < pairs) part[threadIdx.x + k * kMThreads] = v[k];
  csync();
  select_experts<true>(a, part, publish, lane, warp);
}

// ---- hidden layer ------------------------------------------------------------
// How rows lie in the ring, from the plan; the same in both roles.
struct Ring {
  int rb, sb;          // bytes of a row, and of its scales where they travel with it (else 0)
  int stage;           // bytes of a stage: rps rows at `pitch`, then their scales
  int pitch;           // bytes between rows
  int rps;             // rows per stage
  int stages;
  int off;             // where it starts in the tail
};

// The place in the ring, kept by each role across all its rows.
struct RingAt {
  int sl = 0, issued = 0;
  uint32_t ph = 0;
  uint32_t lists = 0;                    // phases of the lists' barriers (the hidden layer's place keeps them)
  __device__ __forceinline__ void next(const Ring& R) { next(R.stages); }
  __device__ __forceinline__ void next(int stages) {
    if (++sl == stages) sl = 0, ph ^= 1u;
  }

};

// A list changes hands both ways: it is written again only after the copying
// warp has read it (a list may be empty, and then nothing else holds the
// computing warps back).
__device__ __forceinline__ void list_free(Smem& sm, const RingAt& at, int i, DevStatus* st) {
  ring_wait(&sm.taken[i], ((at.lists >> i) & 1u) ^ 1u, sm, st, 82);
}
__device__ __forceinline__ void list_written(Smem& sm, RingAt& at, int i) {     // computing warps
  if (threadIdx.x < kBatch) mbar_arrive(&sm.listed[i]);
  at.lists ^= 1u << i;
}
// the number of rows on the list (none, for the whole warp, after a wait that gave up: the
// list may not have been written)
__device__ __forceinline__ int list_wait(Smem& sm, const RingAt& at, int i, const int& n, DevStatus* st) {
  const bool ok = ring_wait(&sm.listed[i], (at.lists >> i) & 1u, sm, st, 77);
  return __all_sync(0xffffffffu, ok) ? *(volatile const int*)&n : 0;
}
__device__ __forceinline__ void list_taken(Smem& sm, RingAt& at, int i, int lane) {
  __syncwarp();
  if (lane == 0) mbar_arrive(&sm.taken[i]);
  at.lists ^= 1u << i;
}

// the copying warp: rows list[0..n), or j0 + i without a list, of matrix w
__device__ __forceinline__ void send_rows(const Ring& R, RingAt& at, Smem& sm, DevStatus* st, const uint8_t* w, const uint8_t* sc,
                                          const int* list, int j0, int n, int lane) {
  for (int i0 = 0; i0 < n; i0 += R.rps) {
    const int nr = min(R.rps, n - i0);
    // (after a give-up nothing more is sent: the last copies' places follow from their number)
    const bool ok = ring_wait(&sm.empty[at.sl], at.ph ^ 1u, sm, st, 74) && !*(volatile int*)&sm.abort;
    if (__all_sync(0xffffffffu, ok)) {
      if (lane == 0) mbar_arrive_expect_tx(&sm.full[at.sl], (uint32_t)(nr * (R.rb + R.sb)));
      __syncwarp();
      unsigned char* dst = sm.tail + R.off + (size_t)at.sl * R.stage;
      for (int r = lane; r < nr; r += 32) {
        const size_t j = (size_t)(list ? list[i0 + r] : j0 + i0 + r);
        bulk_g2s(dst + r * R.pitch, w + j * R.rb, (uint32_t)R.rb, &sm.full[at.sl]);
        if (R.sb && list) bulk_g2s(dst + R.rps * R.pitch + r * R.sb, sc + j * R.sb, (uint32_t)R.sb, &sm.full[at.sl]);
      }
      // (the scales of neighbouring rows in one copy: one of 128 bytes beside each
      // row's 2 KB takes a third of the copies' bandwidth, 5.9 -> 4.1 TB/s)
      if (R.sb && !list && lane == 0)
        bulk_g2s(dst + R.rps * R.pitch, sc + (size_t)(j0 + i0) * R.sb, (uint32_t)(nr * R.sb), &sm.full[at.sl]);
      ++at.issued;
    }
    at.next(R);
  }
}

// bf16 weights: x of up to KU units of 32 values per warp and NG groups of 8
// tokens, four registers per unit and group (a lane's 8 values, in order).
template <int KU, int NG>
struct XFrag {
  uint32_t v[KU][NG][4];
};

// KS warps share the rows' length, the kMWarps / KS groups take the tiles (8 rows, 16 of
// 4-bit weights) in turn.  ku: units of 32 values per warp.
struct Split {
  int ks, groups, part, group, per, n;             // units of this warp: part * per .. + n
  __device__ Split(int d, int ku, int warp) {
    const int units = d / 32;
    ks = 1;
    while (ks * ku < units && ks < kMWarps) ks *= 2;
    groups = kMWarps / ks;
    part = warp % ks;
    group = warp / ks;
    per = (units + ks - 1) / ks;
    n = max(0, min(per, units - part * per));
  }
};

template <int KU, int NG>
__device__ __forceinline__ void load_x(const MoeArgs& a, const Smem& sm, const Split& P, XFrag<KU, NG>& x, int lane) {
  const int g = lane >> 2, q = lane & 3;
#pragma unroll
  for (int n = 0; n < NG; ++n) {
    const int t = sm.tok[n * 8 + g];
    const __nv_bfloat16* px = a.x + (size_t)max(t, 0) * a.d_model + (size_t)P.part * P.per * 32 + q * 8;
#pragma unroll
    for (int i = 0; i < KU; ++i) {
      uint4 v = make_uint4(0, 0, 0, 0);
      if (t >= 0 && i < P.n) v = ld_x(px + i * 32);
      x.v[i][n][0] = v.x, x.v[i][n][1] = v.y, x.v[i][n][2] = v.z, x.v[i][n][3] = v.w;
    }
  }
}

// 4-bit weights: codes become float16 by the conversion instruction, a byte (two
// codes) at a time.  (It runs at a quarter of the rate of simple instructions,
// but moving a code's bits to the exponent and mantissa bits of float16 takes
// four of those a pair, and the warps are short of issue slots; matrix
// instructions of e4m3, into which codes go by two shifts, were three times slower
// than those of float16.)  x, times the power of two that brings its token's
// largest into [2^14, 2^15), is float16, exact down to 2^-39 of that largest.
__device__ __forceinline__ void stage_x(const MoeArgs& a, Smem& sm) {
  const int t = sm.tok[0];
  const float up = sm.xup[t];
  for (int k = threadIdx.x * 8; k < a.d_model; k += kMThreads * 8) {
    const uint4 v = ld_x(a.x + (size_t)t * a.d_model + k);
    const uint32_t u[4] = {v.x, v.y, v.z, v.w};
    uint32_t r[4];
#pragma unroll
    for (int c = 0; c < 4; ++c) {
      const __half2 h = __floats2half2_rn(bf16lo(u[c]) * up, bf16hi(u[c]) * up);
      r[c] = *reinterpret_cast<const uint32_t*>(&h);
    }
    *reinterpret_cast<uint4*>(sm.tail + k * 2) = make_uint4(r[0], r[1], r[2], r[3]);
  }
}

__device__ __forceinline__ void mma_f16(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                        uint32_t b1) {
  asm(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// n rows from the ring times the pass's tokens: sums of row r (of the batch) and
// token t to red[part][r][t].
template <int KU, int NG>
__device__ __forceinline__ void dot_rows_bf16(const MoeArgs& a, const Ring& R, RingAt& at, Smem& sm, const Split& P,
                                              const XFrag<KU, NG>& x, int n, int lane) {
  const int g = lane >> 2, q = lane & 3;
  float* red = sm.red + (size_t)P.part * kBatch * 8;     // kBatch x 8 = 32 x 16
  // the loads of units that the warp does not have repeat its first (x is 0 there)
  const int first = P.n > 0 ? P.part * P.per : 0;
  for (int i0 = 0; i0 < n; i0 += R.rps) {
    const int nr = min(R.rps, n - i0);
    ring_wait(&sm.full[at.sl], at.ph, sm, a.status, 75);
    const unsigned char* stage = sm.tail + R.off + (size_t)at.sl * R.stage;
    for (int t0 = P.group * 8; t0 < nr; t0 += P.groups * 8) {
      const unsigned char* row = stage + (t0 + g < nr ? t0 + g : t0) * R.pitch + first * 64 + q * 16;
      // four sums in turn: one matrix instruction after the other into the
      // same sum takes 20 to 32 cycles each
      constexpr int kSums = 4, kAhead = NG > 1 || KU > 16 ? 4 : 8;
      float acc[kSums][4];
#pragma unroll
      for (int i = 0; i < kSums; ++i)
#pragma unroll
        for (int j = 0; j < 4; ++j) acc[i][j] = 0.0f;
#pragma unroll
      for (int h = 0; h < KU; h += kAhead) {          // kAhead loads before the first product
        uint4 w[kAhead];
#pragma unroll
        for (int i = 0; i < kAhead; ++i) w[i] = *reinterpret_cast<const uint4*>(row + (h + i < P.n ? h + i : 0) * 64);
#pragma unroll
        for (int i = 0; i < kAhead; ++i) {
          const uint32_t(&x0)[4] = x.v[h + i][0];
          const uint32_t(&x1)[4] = x.v[h + i][NG - 1];
          mma_bf16(acc[(2 * i) % kSums], x0[0], NG > 1 ? x1[0] : 0u, x0[1], NG > 1 ? x1[1] : 0u, w[i].x, w[i].y);
          mma_bf16(acc[(2 * i + 1) % kSums], x0[2], NG > 1 ? x1[2] : 0u, x0[3], NG > 1 ? x1[3] : 0u, w[i].z, w[i].w);
        }
      }
#pragma unroll
      for (int i = 1; i < kSums; ++i)
#pragma unroll
        for (int j = 0; j < 4; ++j) acc[0][j] += acc[i][j];
      // tokens g and g + 8, rows 2q and 2q + 1 of the tile
#pragma unroll
      for (int c = 0; c < 2; ++c) {
        const int rr = t0 + 2 * q + c;
        if (rr < nr) {
          red[(i0 + rr) * 8 * NG + g] = acc[0][c];
          if constexpr (NG > 1) red[(i0 + rr) * 8 * NG + 8 + g] = acc[0][2 + c];
        }
      }
    }
    __syncwarp();
    if (lane == 0) mbar_arrive(&sm.empty[at.sl]);
    at.next(R);
  }
}

// 4-bit weights, one token: the neurons are the matrix's 16 rows, the token the first of its
// 8 columns; a unit is one block of 32: its sum times its scale, four blocks at a time (a
// block's second product waits for its first).
__device__ __forceinline__ void dot_rows_fp4(const MoeArgs& a, const Ring& R, RingAt& at, Smem& sm, const Split& P,
                                             const uint8_t* sc, const int* list, int j0, int n, int lane) {
  const int g = lane >> 2, q = lane & 3, first = P.part * P.per, sb = a.d_model / 32;
  float* red = sm.red + (size_t)P.part * kBatch * 8;
  const unsigned char* xs = sm.tail + first * 64 + q * 16;
  const bool whole = R.sb && P.per == 16;             // 16 scales of a row in one load
  int tile = 0;
  for (int i0 = 0; i0 < n; i0 += R.rps) {
    const int nr = min(R.rps, n - i0);
    ring_wait(&sm.full[at.sl], at.ph, sm, a.status, 75);
    const unsigned char* stage = sm.tail + R.off + (size_t)at.sl * R.stage;
    for (int t0 = 0; t0 < nr; t0 += 16, ++tile) {
      if ((tile & (P.groups - 1)) != P.group) continue;
      const int ra = t0 + g < nr ? t0 + g : t0, rc = t0 + 8 + g < nr ? t0 + 8 + g : t0;
      const unsigned char* wa = stage + ra * R.pitch + first * 16 + q * 4;
      const unsigned char* wb = stage + rc * R.pitch + first * 16 + q * 4;
      const uint8_t *pa, *pb;                         // the blocks' scales
      uint4 ca = make_uint4(0, 0, 0, 0), cb = ca;
      if (R.sb) {
        pa = stage + R.rps * R.pitch + ra * R.sb + first;
        pb = stage + R.rps * R.pitch + rc * R.sb + first;
        if (whole) ca = *reinterpret_cast<const uint4*>(pa), cb = *reinterpret_cast<const uint4*>(pb);
      } else {
        pa = sc + (size_t)(list ? list[i0 + ra] : j0 + i0 + ra) * sb + first;
        pb = sc + (size_t)(list ? list[i0 + rc] : j0 + i0 + rc) * sb + first;
      }
      float acc[2] = {0.0f, 0.0f};
#pragma unroll
      for (int h = 0; h < 16; h += 4) {
        if (h >= P.n) break;
        uint32_t sa, sbw, va[4], vb[4];
        uint4 x[4];
        if (whole) {
          sa = h == 0 ? ca.x : h == 4 ? ca.y : h == 8 ? ca.z : ca.w;
          sbw = h == 0 ? cb.x : h == 4 ? cb.y : h == 8 ? cb.z : cb.w;
        } else {
          sa = sbw = 0;
#pragma unroll
          for (int i = 0; i < 4; ++i)
            if (h + i < P.n) {
              sa |= (uint32_t)(R.sb ? pa[h + i] : __ldg(pa + h + i)) << (8 * i);
              sbw |= (uint32_t)(R.sb ? pb[h + i] : __ldg(pb + h + i)) << (8 * i);
            }
        }
#pragma unroll
        for (int i = 0; i < 4; ++i) {                 // (units behind the warp's last have x = 0)
          const int k = h + i < P.n ? h + i : h;
          va[i] = *reinterpret_cast<const uint32_t*>(wa + k * 16);
          vb[i] = *reinterpret_cast<const uint32_t*>(wb + k * 16);
          x[i] = g == 0 && h + i < P.n ? *reinterpret_cast<const uint4*>(xs + k * 64) : make_uint4(0, 0, 0, 0);
        }
        float d[4][4];
        uint32_t ha[4][4], hb[4][4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          d[i][0] = d[i][1] = d[i][2] = d[i][3] = 0.0f;
          e2m1x8_to_half2(va[i], ha[i]);
          e2m1x8_to_half2(vb[i], hb[i]);
          mma_f16(d[i], ha[i][0], hb[i][0], ha[i][1], hb[i][1], x[i].x, x[i].y);
        }
#pragma unroll
        for (int i = 0; i < 4; ++i) mma_f16(d[i], ha[i][2], hb[i][2], ha[i][3], hb[i][3], x[i].z, x[i].w);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          // (the least scale, 2^-127, is the subnormal number below them; 255 counts as an
          // infinity, which makes a NaN of its codes, all 0)
          acc[0] = fmaf(d[i][0], __uint_as_float(max(((sa >> (8 * i)) & 0xffu) << 23, 0x400000u)), acc[0]);
          acc[1] = fmaf(d[i][2], __uint_as_float(max(((sbw >> (8 * i)) & 0xffu) << 23, 0x400000u)), acc[1]);
        }
      }
      // rows g and g + 8 of the tile
      float* o = red + (size_t)(i0 + t0 + g) * 8;
      if (q == 0 && t0 + g < nr) o[0] = acc[0];
      if (q == 0 && t0 + 8 + g < nr) o[64] = acc[1];
    }
    __syncwarp();
    if (lane == 0) mbar_arrive(&sm.empty[at.sl]);
    at.next(R);
  }
}

// One token, d_model <= 4096: the CTA goes on to its neurons' down rows, kVec
// vectors of 8 columns per thread.
constexpr int kVec = 4096 / (kMThreads * 8);
template <bool FP4>
__device__ __forceinline__ void down_stage_rows(const MoeArgs& a, const Ring& R, RingAt& at, Smem& sm, const uint8_t* sc,
                                                const int* list, const float* val, int n, float (&y)[kVec][8], int lane) {
  const int tid = threadIdx.x;
  for (int i0 = 0; i0 < n; i0 += R.rps) {
    const int nr = min(R.rps, n - i0);
    ring_wait(&sm.full[at.sl], at.ph, sm, a.status, 76);
    const unsigned char* stage = sm.tail + R.off + (size_t)at.sl * R.stage;
#pragma unroll 4
    for (int r = 0; r < nr; ++r) {
      const unsigned char* row = stage + r * R.pitch;
      const float h = val[i0 + r];
#pragma unroll
      for (int v = 0; v < kVec; ++v) {
        const int col = (v * kMThreads + tid) * 8;
        if (col >= a.d_model) break;
        if constexpr (!FP4) {
          const uint4 w = *reinterpret_cast<const uint4*>(row + col * 2);
          const uint32_t u[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
          for (int c = 0; c < 4; ++c) {
            y[v][2 * c] = fmaf(h, bf16lo(u[c]), y[v][2 * c]);
            y[v][2 * c + 1] = fmaf(h, bf16hi(u[c]), y[v][2 * c + 1]);
          }
        } else {
          const uint32_t b = R.sb ? stage[R.rps * R.pitch + r * R.sb + col / 32]
                                  : __ldg(sc + (size_t)list[i0 + r] * (a.d_model / 32) + col / 32);
          const float hs = h * e8m0_value(b);
          uint32_t f[4];
          e2m1x8_to_half2(*reinterpret_cast<const uint32_t*>(row + col / 2), f);
#pragma unroll
          for (int c = 0; c < 4; ++c) {
            const float2 e = __half22float2(*reinterpret_cast<const __half2*>(&f[c]));
            y[v][2 * c] = fmaf(hs, e.x, y[v][2 * c]);
            y[v][2 * c + 1] = fmaf(hs, e.y, y[v][2 * c + 1]);
          }
        }
      }
    }
    __syncwarp();
    if (lane == 0) mbar_arrive(&sm.empty[at.sl]);
    at.next(R);
  }
}

// one token: the share of the choice whose slot this is
__device__ __forceinline__ float choice_share(const MoeArgs& a, const Smem& sm, int slot) {
  float p = 0.0f;
  for (int j = 0; j < a.top_k; ++j)
    if (sm.slot[j] == slot) p = sm.share[j];
  return p;
}

// A run: neurons [j0, j1) of active expert ai for nt of its tokens, whose slots
// start at slot0.  Both roles go through the same batches.
struct Run {
  int ai, e, slot0, nt, j0, j1, batch;
  bool add;            // not the first pass over these neurons: flags are only set
  bool keep_zeros;     // another pass may open a neuron that this one closes: its h is written too
};

struct ExpertMats {
  const uint8_t *w1, *w2, *wd, *s1, *s2, *sd;
};
template <bool FP4>
__device__ __forceinline__ ExpertMats expert_mats(const MoeArgs& a, int e) {
  const size_t mat = (size_t)a.d_ff * a.d_model, wo = FP4 ? (size_t)e * (mat / 2) : (size_t)e * mat * 2;
  const size_t so = FP4 ? (size_t)e * (mat / 32) : 0;
  return ExpertMats{a.w1 + wo, a.w2 + wo, a.wd + wo, FP4 ? a.s1 + so : nullptr, FP4 ? a.s2 + so : nullptr,
                    FP4 ? a.sd + so : nullptr};
}

template <bool FP4, bool ONE>
__device__ void send_run(const MoeArgs& a, const Ring& R, RingAt& at, Smem& sm, const Run& u, int lane) {
  const ExpertMats M = expert_mats<FP4>(a, u.e);
  const int nb = (u.j1 - u.j0 + u.batch - 1) / u.batch;
  for (int b = 0; b < nb + (ONE ? 2 : 1); ++b) {
    if (b < nb) {
      const int jb = u.j0 + b * u.batch;
      send_rows(R, at, sm, a.status, M.w1, M.s1, nullptr, jb, min(u.batch, u.j1 - jb), lane);
    }
    if (b >= 1 && b - 1 < nb) {
      const int s = (b - 1) & 1;
      const int n = list_wait(sm, at, s, sm.nrows[s], a.status);
      send_rows(R, at, sm, a.status, M.w2, M.s2, sm.rows[s], 0, n, lane);
      list_taken(sm, at, s, lane);
    }
    if (ONE && b >= 2) {
      const int s = b & 1;
      const int n = list_wait(sm, at, 2 + s, sm.ndrows[s], a.status);
      send_rows(R, at, sm, a.status, M.wd, M.sd, sm.drows[s], 0, n, lane);
      list_taken(sm, at, 2 + s, lane);
    }
  }
}

// the sum at place i (row * 8 NG + token) over the warps that share the rows
__device__ __forceinline__ float dot_sum(const Smem& sm, const Split& P, int i) {
  float v = 0.0f;
#pragma unroll 4
  for (int k = 0; k < P.ks; ++k) v += sm.red[(size_t)k * kBatch * 8 + i];
  return v;
}

template <bool FP4, int KU, int NG, bool ONE>
__device__ __forceinline__ void compute_run(const MoeArgs& a, const Ring& R, RingAt& at, Smem& sm, const Run& u,
                                            float (&y)[kVec][8], int lane, int warp) {
  const int tid = threadIdx.x;
  const ExpertMats M = expert_mats<FP4>(a, u.e);
  const float* b1 = a.b1 ? a.b1 + (size_t)u.e * a.d_ff : nullptr;
  const float* b2 = a.b2 ? a.b2 + (size_t)u.e * a.d_ff : nullptr;
  const Split P(a.d_model, KU, warp);
  XFrag<FP4 ? 1 : KU, NG> x;
  if constexpr (FP4) {
    stage_x(a, sm);
    csync();
  } else {
    load_x<KU, NG>(a, sm, P, x, lane);
  }
  const int nb = (u.j1 - u.j0 + u.batch - 1) / u.batch;
  // this thread's places in a batch's results: i = tid and tid + 256, row
  // i / 8 NG, token i % 8 NG (the same for both)
  constexpr int kPer = kBatch * 8 / kMThreads, kTok = 8 * NG, kRowsPerWarp = 32 / kTok;
  const int c = tid % kTok, r0 = tid / kTok;
  constexpr int kStep = kMThreads / kTok;                // rows between a thread's places
  const float back = FP4 && c < u.nt ? 1.0f / sm.xup[sm.tok[c]] : 1.0f;
  const float share = ONE ? choice_share(a, sm, u.slot0) : 0.0f;
  for (int b = 0; b < nb + (ONE ? 2 : 1); ++b) {
    // (one body for both factors: the code of two does not stay in the
    // instruction cache)
#pragma unroll 1
    for (int second = 0; second < 2; ++second) {
      const int bb = b - second;
      if (bb < 0 || bb >= nb) continue;
      const int s = bb & 1, jb = u.j0 + bb * u.batch;
      const int n = second ? sm.nrows[s] : min(u.batch, u.j1 - jb);
      const int* list = second ? sm.rows[s] : nullptr;
      const float* bs = second ? b2 : b1;
      int j[kPer];
      float bias[kPer];
#pragma unroll
      for (int k = 0; k < kPer; ++k) {
        const int r = r0 + k * kStep;
        j[k] = r < n ? (list ? list[r] : jb + r) : -1;
        bias[k] = bs && j[k] >= 0 ? __ldg(bs + j[k]) : 0.0f;
      }
      if constexpr (FP4) dot_rows_fp4(a, R, at, sm, P, second ? M.s2 : M.s1, list, jb, n, lane);
      else dot_rows_bf16<KU, NG>(a, R, at, sm, P, x, n, lane);
      csync();
      if (!second) {
        // first factors of batch b, and its open neurons
#pragma unroll
        for (int k = 0; k < kPer; ++k) {
          float v = 0.0f;
          if (j[k] >= 0 && c < u.nt) {
            v = relu_nan(dot_sum(sm, P, tid + k * kMThreads) * back + bias[k]);
            if (!a.drelu) v *= v;
          }
          sm.first[s][tid + k * kMThreads] = v;
          const unsigned any = __ballot_sync(0xffffffffu, v != 0.0f);
          if (lane == 0) {
            uint32_t m = 0;
#pragma unroll
            for (int i = 0; i < kRowsPerWarp; ++i)
              if ((any >> (i * kTok)) & ((1u << kTok) - 1u)) m |= 1u << i;
            sm.mask[k * kMWarps + warp] = m;
          }
        }
        csync();
        list_free(sm, at, s, a.status);
        if (tid < kBatch) {
          // row tid of the batch (rows behind n are closed)
          uint64_t m = 0;
#pragma unroll
          for (int w = 0; w < kPer * kMWarps; ++w) m |= (uint64_t)sm.mask[w] << (w * kRowsPerWarp);
          const bool open = (m >> tid) & 1u;
          if (open) sm.rows[s][__popcll(m & ((1ull << tid) - 1ull))] = jb + tid;
          if (tid == 0) sm.nrows[s] = __popcll(m);
          if constexpr (!ONE) {
            // a closed neuron's h is 0 and is not read again: only its flag is
            // written (unless another pass's tokens may open it)
            if (!open && tid < n) {
              if (!u.add) a.nz[(size_t)u.ai * a.d_ff + jb + tid] = 0;
              if (u.keep_zeros)
                for (int t = 0; t < u.nt; ++t) __stcg(a.h + (size_t)(u.slot0 + t) * a.d_ff + jb + tid, 0.0f);
            }
          }
        }
        list_written(sm, at, s);
        csync();
        continue;
      }
      // second factors of the open neurons, and h
#pragma unroll
      for (int k = 0; k < kPer; ++k) {
        float h = 0.0f;
        if (j[k] >= 0 && c < u.nt) {
          float v = dot_sum(sm, P, tid + k * kMThreads) * back + bias[k];
          if (a.drelu) v = relu_nan(v);
          // (a closed first factor is 0 whatever the other is: another token has opened the neuron)
          const float f = sm.first[s][(j[k] - jb) * kTok + c];
          h = f == 0.0f ? 0.0f : f * v;
          if constexpr (!ONE) __stcg(a.h + (size_t)(u.slot0 + c) * a.d_ff + j[k], h);
        }
        if constexpr (!ONE) {
          const unsigned any = __ballot_sync(0xffffffffu, h != 0.0f);
          const unsigned mine = (any >> (lane / kTok * kTok)) & ((1u << kTok) - 1u);
          if (j[k] >= 0 && c == 0) {
            uint8_t* f = a.nz + (size_t)u.ai * a.d_ff + j[k];
            if (u.add) { if (mine) *f = 1; }
            else *f = mine != 0;
          }
        } else if (c == 0) {
          sm.hval[r0 + k * kStep] = h;
        }
      }
      csync();
      if constexpr (ONE) {
        list_free(sm, at, 2 + s, a.status);
        if (tid < kBatch) {
          // the neurons with h != 0, in order, and p h
          const float hv = tid < n ? sm.hval[tid] : 0.0f;
          const unsigned m = __ballot_sync(0xffffffffu, hv != 0.0f);
          if (lane == 0) sm.scan[warp] = __popc(m);
          asm volatile("bar.sync 2, 64;" ::: "memory");
          if (hv != 0.0f) {
            const int at2 = (warp ? sm.scan[0] : 0) + __popc(m & lanemask_lt());
            sm.drows[s][at2] = sm.rows[s][tid];
            sm.dval[s][at2] = hv * share;
          }
          if (tid == 0) sm.ndrows[s] = sm.scan[0] + sm.scan[1];
        }
        list_written(sm, at, 2 + s);
        csync();
      }
    }
    if (ONE && b >= 2) {
      const int s = b & 1;
      down_stage_rows<FP4>(a, R, at, sm, M.sd, sm.drows[s], sm.dval[s], sm.ndrows[s], y, lane);
    }
  }
}

// The runs of a hidden-layer item, in the order both roles take them: f(run).
// The items have equal shares of the neurons times their experts' passes.
template <typename F>
__device__ __forceinline__ void each_run(const MoeArgs& a, const Smem& sm, int item, int pass, F&& f) {
  const long long N = (long long)sm.cum[0][sm.active] * a.d_ff;
  const long long n0 = N * item / a.plan.hidden_items, n1 = N * (item + 1) / a.plan.hidden_items;
  // the first expert of the range
  int ai = 0;
  for (int step = kMoeMaxE / 2; step; step >>= 1)
    if (ai + step < sm.active && (long long)sm.cum[0][ai + step] * a.d_ff <= n0) ai += step;
  for (; ai < sm.active; ++ai) {
    const long long at = (long long)sm.cum[0][ai] * a.d_ff;
    if (at >= n1) break;
    const int np = passes_of(sm, 0, ai);
    const long long lo = max(n0 - at, 0ll), hi = min(n1 - at, (long long)np * a.d_ff);
    Run u;
    u.ai = ai;
    u.j0 = (int)(lo / np);
    u.j1 = (int)(hi / np);
    if (hi <= 0 || u.j0 >= u.j1) continue;
    u.e = sm.expert[ai];
    const int cnt = sm.count[ai], first = sm.firsts[ai];
    // (every pass over a batch's worth of neurons before the next, so that the
    // second pass finds the rows in L2)
    const int step = cnt > pass ? 2 * kBatch : u.j1 - u.j0;
    const int end = u.j1;
    for (int j = u.j0; j < end; j += step)
      for (int t0 = 0; t0 < cnt; t0 += pass) {
        Run v = u;
        v.j0 = j;
        v.j1 = min(end, j + step);
        v.slot0 = first + t0;
        v.nt = min(pass, cnt - t0);
        // batches of about the same size, whole tiles of 16
        const int most = v.nt > 8 ? kBatch / 2 : kBatch, n = v.j1 - v.j0, nb = (n + most - 1) / most;
        v.batch = min(most, ((n + nb - 1) / nb + 15) / 16 * 16);
        v.add = t0 > 0;
        v.keep_zeros = cnt > pass;
        f(v);
      }
  }
}

// tokens of a run into sm.tok (computing warps)
__device__ __forceinline__ void run_tokens(Smem& sm, const Run& u) {
  csync();
  if (threadIdx.x < 8 * kMaxNg) sm.tok[threadIdx.x] = (int)threadIdx.x < u.nt ? sm.token[u.slot0 + threadIdx.x] : -1;
  csync();
}

// (a function of its own per instance: inlined together they share the
// registers of the largest and spill)
template <int KU, int NG>
__device__ __noinline__ void compute_pass(const MoeArgs& a, const Ring& R, RingAt& at, const Run& u, int lane, int warp) {
  Smem& sm = smem();
  float none[kVec][8];
  RingAt here = at;                     // in registers
  const Ring ring = R;
  const Run run = u;
  compute_run<false, KU, NG, false>(a, ring, here, sm, run, none, lane, warp);
  at = here;
}

// units of 32 values per warp: bf16, d_model <= 4096: all of them in registers
constexpr int kUnits = 16;

template <bool FP4, bool ONE>
__device__ __forceinline__ void hidden_item(const MoeArgs& a, const Ring& R, RingAt& at, Smem& sm, int item, int lane,
                                            int warp) {
  const int pass = a.plan.hidden_tokens;
  if (warp == kMWarps) {
    each_run(a, sm, item, pass, [&](const Run& u) { send_run<FP4, ONE>(a, R, at, sm, u, lane); });
    return;
  }
  float y[kVec][8];
  if constexpr (ONE) {
#pragma unroll
    for (int v = 0; v < kVec; ++v)
#pragma unroll
      for (int i = 0; i < 8; ++i) y[v][i] = 0.0f;
  }
  each_run(a, sm, item, pass, [&](const Run& u) {
    run_tokens(sm, u);
    if constexpr (ONE) {
      compute_run<FP4, kUnits, 1, true>(a, R, at, sm, u, y, lane, warp);
    } else {
      if (a.d_model > 4096) compute_pass<2 * kUnits, 1>(a, R, at, u, lane, warp);
      else if (u.nt <= 8) compute_pass<kUnits, 1>(a, R, at, u, lane, warp);
      else compute_pass<kUnits, 2>(a, R, at, u, lane, warp);
    }
  });
  if constexpr (ONE) {
#pragma unroll
    for (int v = 0; v < kVec; ++v) {
      const int col = (v * kMThreads + threadIdx.x) * 8;
      if (col < a.d_model) {
        float* o = a.parts + (size_t)item * a.d_model + col;
        __stcg(reinterpret_cast<float4*>(o), make_float4(y[v][0], y[v][1], y[v][2], y[v][3]));
        __stcg(reinterpret_cast<float4*>(o + 4), make_float4(y[v][4], y[v][5], y[v][6], y[v][7]));
      }
    }
  }
}

// ---- down projection ---------------------------------------------------------
// Item: (expert, column tile, range of neurons).  The range's flagged neurons
// are listed, 8 per thread at a time; the tile's piece of their down rows comes
// through the ring 16 neurons per stage (one step of the matrix instructions);
// their h is staged as three bf16 numbers, 128 neurons at a time.  A warp has
// STR strips of 64 columns, in turn over the warps.
struct DownItem {
  int ai, e, s, j0, j1, c0, cw;          // columns [c0, c0 + cw)
};
// Its stages are others than the hidden layer's, in the same memory, with
// barriers of their own (an item begins and ends with every stage free).
struct DownRing {
  int pb;                                // bytes of a piece
  int pitch, stages, off;
};
constexpr int kRowsStage = 16;

// splits of an expert's neurons: S per pass over them, about one item per CTA in
// all; the buffers hold max_splits
__device__ __forceinline__ int down_splits(const MoeArgs& a, const Smem& sm) {
  const int s = a.plan.grid / (sm.cum[1][sm.active] * a.plan.col_tiles);
  return max(1, s);
}
__device__ __forceinline__ int expert_splits(const MoeArgs& a, const Smem& sm, int ai, int S) {
  return min(S * passes_of(sm, 1, ai), a.plan.max_splits);
}
__device__ __forceinline__ int down_items(const MoeArgs& a, const Smem& sm, int S) {
  int n = 0;
  for (int ai = 0; ai < sm.active; ++ai) n += expert_splits(a, sm, ai, S);
  return n * a.plan.col_tiles;
}

__device__ __forceinline__ DownItem down_place(const MoeArgs& a, const Smem& sm, int item, int S) {
  DownItem d;
  int rest = item / a.plan.col_tiles, n = expert_splits(a, sm, 0, S);
  for (d.ai = 0; rest >= n; n = expert_splits(a, sm, ++d.ai, S)) rest -= n;
  d.s = rest;
  d.e = sm.expert[d.ai];
  // whole groups of 8 neurons (their flags are read 8 at a time)
  d.j0 = (int)((long long)(a.d_ff / 8) * d.s / n) * 8;
  d.j1 = (int)((long long)(a.d_ff / 8) * (d.s + 1) / n) * 8;
  d.c0 = item % a.plan.col_tiles * a.plan.tile_cols;
  d.cw = min(a.plan.tile_cols, a.d_model - d.c0);
  return d;
}
__device__ __forceinline__ DownRing down_ring(const MoeArgs& a, const DownItem& d) {
  DownRing r;
  r.pb = d.cw * 2;
  r.pitch = a.plan.down_pitch;
  r.stages = a.plan.down_stages;
  r.off = 0;
  return r;
}

__device__ void send_down(const MoeArgs& a, RingAt& at, Smem& sm, const DownItem& d, int passes, int lane) {
  const DownRing R = down_ring(a, d);
  const size_t rb = (size_t)a.d_model * 2;
  const uint8_t* w = a.wd + (size_t)d.e * a.d_ff * rb + d.c0 * 2;
  for (int p = 0; p < passes; ++p)
    for (int jl = d.j0; jl < d.j1; jl += kListD) {
      const int total = list_wait(sm, at, 2, sm.ndrows[0], a.status);
      for (int i0 = 0; i0 < total; i0 += kRowsStage) {
        const int nr = min(kRowsStage, total - i0);
        const bool ok = ring_wait(&sm.dempty[at.sl], at.ph ^ 1u, sm, a.status, 80) && !*(volatile int*)&sm.abort;
        if (__all_sync(0xffffffffu, ok)) {
          if (lane == 0) mbar_arrive_expect_tx(&sm.dfull[at.sl], (uint32_t)(nr * R.pb));
          __syncwarp();
          unsigned char* dst = sm.tail + R.off + (size_t)at.sl * kRowsStage * R.pitch;
          if (lane < nr) {
            const size_t j = (size_t)(jl + sm.d.list[i0 + lane]);
            bulk_g2s(dst + lane * R.pitch, w + j * rb, (uint32_t)R.pb, &sm.dfull[at.sl]);
          }
          ++at.issued;
        }
        at.next(R.stages);
      }
      list_taken(sm, at, 2, lane);
    }
}

template <int NG, int STR>
__device__ __noinline__ void down_rows(const MoeArgs& a, RingAt& at_, const DownItem& d_, int slot0, int nt, int lane, int warp) {
  Smem& sm = smem();
  RingAt at = at_;
  const DownItem d = d_;
  const DownRing R = down_ring(a, d);
  constexpr int kCols = 8;                           // columns of a lane
  constexpr int kMma = kCols / 2;                    // MMAs per 16 neurons and token group
  const int g = lane >> 2, q = lane & 3, tid = threadIdx.x;
  int col[STR];
#pragma unroll
  for (int x = 0; x < STR; ++x) col[x] = (x * kMWarps + warp) * (8 * kCols) + g * kCols;
  float acc[STR][kMma][NG][4];
#pragma unroll
  for (int x = 0; x < STR; ++x)
#pragma unroll
    for (int m = 0; m < kMma; ++m)
#pragma unroll
      for (int n = 0; n < NG; ++n)
#pragma unroll
        for (int i = 0; i < 4; ++i) acc[x][m][n][i] = 0.0f;

  for (int jl = d.j0; jl < d.j1; jl += kListD) {
    // list the flagged neurons of this round, in order: 8 flags per thread
    const int jt = jl + tid * 8;
    uint2 f8 = make_uint2(0, 0);
    if (jt < min(d.j1, jl + kListD)) f8 = __ldcg(reinterpret_cast<const uint2*>(a.nz + (size_t)d.ai * a.d_ff + jt));
    uint32_t bits8 = 0;
#pragma unroll
    for (int i = 0; i < 8; ++i) bits8 |= (((i < 4 ? f8.x : f8.y) >> (8 * (i & 3))) & 1u) << i;
    const int cnt = __popc(bits8);
    int inc = cnt;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int up = __shfl_up_sync(0xffffffffu, inc, o);
      if (lane >= o) inc += up;
    }
    list_free(sm, at, 2, a.status);
    csync();                                         // the previous round's list and h are read
    if (lane == 31) sm.scan[warp] = inc;
    csync();
    int at2 = inc - cnt, total = 0;
#pragma unroll
    for (int v = 0; v < kMWarps; ++v) {
      if (v < warp) at2 += sm.scan[v];
      total += sm.scan[v];
    }
    for (uint32_t m = bits8; m; m &= m - 1u) sm.d.list[at2++] = (uint16_t)(tid * 8 + __ffs((int)m) - 1);
    if (tid == 0) sm.ndrows[0] = total;
    csync();
    list_written(sm, at, 2);
    for (int l0 = 0; l0 < total; l0 += kRowsD) {
      const int n = min(kRowsD, total - l0), np = (n + 15) & ~15;
      if (l0) csync();                               // the previous neurons' h is read
      // h of these neurons as three bf16 numbers; neuron r of a step of 16 is
      // lane quarter r % 4's r / 4-th
      for (int i = tid; i < np * 8 * NG; i += kMThreads) {
        const int r = i % np, c = i / np;
        float h = 0.0f;
        if (r < n && c < nt) h = __ldcg(a.h + (size_t)(slot0 + c) * a.d_ff + jl + sm.d.list[l0 + r]);
        // (an infinity or a NaN has no rest)
        const bool finite = fabsf(h) <= 3.0e38f;
        const int to = c * kHPitch + (r & ~15) + (r & 3) * 4 + ((r & 15) >> 2);
#pragma unroll
        for (int v = 0; v < 3; ++v) {
          const __nv_bfloat16 b = __float2bfloat16_rn(h);
          sm.d.h[v][to] = b;
          h = finite ? h - __bfloat162float(b) : 0.0f;
        }
      }
      csync();
      for (int st = 0; st < np / 16; ++st) {
        const int nr = min(kRowsStage, n - st * 16);
        ring_wait(&sm.dfull[at.sl], at.ph, sm, a.status, 81);
        const unsigned char* stage = sm.tail + R.off + (size_t)at.sl * kRowsStage * R.pitch;
        // this lane's rows 4 i + q (rows that the stage does not have repeat the
        // first: their h is 0)
        const unsigned char* row[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) row[i] = stage + (4 * i + q < nr ? 4 * i + q : 0) * R.pitch;
        uint2 b[NG][3];
#pragma unroll
        for (int t = 0; t < NG; ++t)
#pragma unroll
          for (int v = 0; v < 3; ++v)
            b[t][v] = *reinterpret_cast<const uint2*>(sm.d.h[v] + (t * 8 + g) * kHPitch + st * 16 + 4 * q);
#pragma unroll
        for (int x = 0; x < STR; ++x) {
          if ((x * kMWarps + warp) * (8 * kCols) >= d.cw) break;          // whole warps: the strip does not exist
          const int cl = col[x] < d.cw ? col[x] : 0;
          auto mmas = [&](int m, uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3) {
#pragma unroll
            for (int t = 0; t < NG; ++t)
#pragma unroll
              for (int v = 0; v < 3; ++v) mma_bf16(acc[x][m][t], a0, a1, a2, a3, b[t][v].x, b[t][v].y);
          };
          uint4 u[4];
#pragma unroll
          for (int i = 0; i < 4; ++i) u[i] = *reinterpret_cast<const uint4*>(row[i] + cl * 2);
          const uint32_t* u0 = reinterpret_cast<const uint32_t*>(&u[0]);
          const uint32_t* u1 = reinterpret_cast<const uint32_t*>(&u[1]);
          const uint32_t* u2 = reinterpret_cast<const uint32_t*>(&u[2]);
          const uint32_t* u3 = reinterpret_cast<const uint32_t*>(&u[3]);
#pragma unroll
          for (int m = 0; m < kMma; ++m)
            mmas(m, __byte_perm(u0[m], u1[m], 0x5410), __byte_perm(u0[m], u1[m], 0x7632),
                 __byte_perm(u2[m], u3[m], 0x5410), __byte_perm(u2[m], u3[m], 0x7632));
        }
        __syncwarp();
        if (lane == 0) mbar_arrive(&sm.dempty[at.sl]);
        at.next(R.stages);
      }
    }
  }
  const size_t slots = (size_t)a.T * a.top_k;
#pragma unroll
  for (int x = 0; x < STR; ++x) {
    if (col[x] >= d.cw) continue;
#pragma unroll
    for (int t = 0; t < NG; ++t)
#pragma unroll
      for (int c = 0; c < 2; ++c) {
        const int n = t * 8 + 2 * q + c;
        if (n < nt) {
          float* o = a.parts + ((size_t)d.s * slots + slot0 + n) * a.d_model + d.c0 + col[x];
#pragma unroll
          for (int m = 0; m < kMma; m += 2)
            __stcg(reinterpret_cast<float4*>(o + 2 * m),
                   make_float4(acc[x][m][t][c], acc[x][m][t][2 + c], acc[x][m + 1][t][c], acc[x][m + 1][t][2 + c]));
        }
      }
  }
  at_ = at;
}

// strips per warp: with at most 8 tokens their sums take 64 registers, with 16
// half the strips do
constexpr int kStrips = 4;

__device__ void down_item(const MoeArgs& a, RingAt& at, Smem& sm, int item, int S, int lane, int warp) {
  const DownItem d = down_place(a, sm, item, S);
  const int first = sm.firsts[d.ai], cnt = sm.count[d.ai], pass = a.plan.down_tokens;
  if (warp == kMWarps) {
    send_down(a, at, sm, d, (cnt + pass - 1) / pass, lane);
    return;
  }
  for (int t0 = 0; t0 < cnt; t0 += pass) {
    const int nt = min(pass, cnt - t0);
    if (pass == 8) down_rows<1, kStrips>(a, at, d, first + t0, nt, lane, warp);
    else if (nt <= 8) down_rows<1, kStrips / 2>(a, at, d, first + t0, nt, lane, warp);
    else down_rows<2, kStrips / 2>(a, at, d, first + t0, nt, lane, warp);
  }
}

// ---- sums ----------------------------------------------------------------------
// 16 vectors of 4 outputs per item; kMThreads / 16
// threads share the partial sums of each (in turn), so that their loads are all in flight at once
__device__ void sum_item(const MoeArgs& a, Smem& sm, int item, int S) {
  const int n4 = a.d_model / 4, tid = threadIdx.x, vec = tid & 15, part = tid >> 4;
  for (long long i0 = (long long)item * 16; i0 < (long long)a.T * n4; i0 += (long long)a.plan.out_items * 16) {
  const long long i = i0 + vec;
  const bool ok = i < (long long)a.T * n4;
  const int t = ok ? (int)(i / n4) : 0, c = ok ? (int)(i - (long long)t * n4) * 4 : 0;
  const size_t slots = (size_t)a.T * a.top_k;
  float4 y = make_float4(0, 0, 0, 0);
  if (ok) {
    if (a.plan.one_token) {
      const float* src = a.parts + c;
#pragma unroll 8
      for (int s = part; s < a.plan.hidden_items; s += kMThreads / 16) {
        const float4 u = __ldcg(reinterpret_cast<const float4*>(src + (size_t)s * a.d_model));
        y.x += u.x, y.y += u.y, y.z += u.z, y.w += u.w;
      }
    } else {
      for (int j = 0; j < a.top_k; ++j) {
        const int slot = sm.slot[t * a.top_k + j];
        const float p = sm.share[t * a.top_k + j];
        const float* src = a.parts + (size_t)slot * a.d_model + c;
        const int n = expert_splits(a, sm, sm.slot_expert[slot], S);
#pragma unroll 4
        for (int s = part; s < n; s += kMThreads / 16) {
          const float4 u = __ldcg(reinterpret_cast<const float4*>(src + (size_t)s * slots * a.d_model));
          y.x = fmaf(p, u.x, y.x), y.y = fmaf(p, u.y, y.y), y.z = fmaf(p, u.z, y.z), y.w = fmaf(p, u.w, y.w);
        }
      }
    }
  }
  float4* red = reinterpret_cast<float4*>(sm.red);
  csync();
  red[tid] = y;
  csync();
  if (part == 0 && ok) {
    for (int k = 1; k < kMThreads / 16; ++k) {
      const float4 u = red[k * 16 + vec];
      y.x += u.x, y.y += u.y, y.z += u.z, y.w += u.w;
    }
    const size_t o = (size_t)t * a.d_model + c;
    if (a.y_bf16) {
      uint2 b;
      b.x = (uint32_t)f32_to_bf16_bits(y.x) | ((uint32_t)f32_to_bf16_bits(y.y) << 16);
      b.y = (uint32_t)f32_to_bf16_bits(y.z) | ((uint32_t)f32_to_bf16_bits(y.w) << 16);
      *reinterpret_cast<uint2*>(reinterpret_cast<__nv_bfloat16*>(a.y) + o) = b;
    } else {
      *reinterpret_cast<float4*>(reinterpret_cast<float*>(a.y) + o) = y;
    }
  }
  }
}

// ---- ahead of the tensor-core products (4-bit weights) ---------------------------
// x as eight 4-bit numbers (moe_fp4_factors.cu): 8 values per thread, the four
// threads of a block share its largest magnitude.
__device__ void split_x(const MoeArgs& a, size_t v) {
  const size_t n8 = (size_t)a.T * a.d_model / 8;
  const uint32_t per = (uint32_t)a.d_model / 8, t = (uint32_t)v / per, at = (uint32_t)v - t * per;
  float r[8] = {0.0f, 0.0f, 0.0f, 0.0f, 0.0f, 0.0f, 0.0f, 0.0f};
  if (v < n8) {
    const uint4 u = ld_x(a.x + v * 8);
    const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) r[2 * i] = bf16lo(w[i]), r[2 * i + 1] = bf16hi(w[i]);
  }
  uint32_t m = 0;
#pragma unroll
  for (int i = 0; i < 8; ++i) m = max(m, __float_as_uint(r[i]) & 0x7fffffffu);
  m = max(m, __shfl_xor_sync(0xffffffffu, m, 1));
  m = max(m, __shfl_xor_sync(0xffffffffu, m, 2));
  if (v >= n8) return;
  const bool finite = m < 0x7f800000u;
  const int first = finite ? max((int)(m >> 23) - 1, 0) : 255;
  if ((threadIdx.x & 3) == 0) a.xs[(size_t)t * moe_xs_pitch(a.d_model) + at / 4] = (uint8_t)first;
  uint32_t* out = reinterpret_cast<uint32_t*>(a.xt) + (size_t)t * kMoeXTerms * per + at;
#pragma unroll
  for (int i = 0; i < kMoeXTerms; ++i) {
    const uint32_t s = (uint32_t)max(first - 3 * i, 0);
    const float inv = finite ? __uint_as_float((254u - s) << 23) : 0.0f, back = e8m0_value(s);
    float q[8];
#pragma unroll
    for (int k = 0; k < 8; ++k) q[k] = finite ? r[k] * inv : 0.0f;
    const uint32_t c = e2m1x8(q);
    out[(size_t)i * per] = c;
    uint32_t h[4];
    e2m1x8_to_half2(c, h);
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      const float2 e = __half22float2(*reinterpret_cast<const __half2*>(&h[k]));
      r[2 * k] = fmaf(-e.x, back, r[2 * k]);
      r[2 * k + 1] = fmaf(-e.y, back, r[2 * k + 1]);
    }
  }
}

// Blocks: the router's, of which the last to finish selects; x's terms.
__global__ void __launch_bounds__(kMThreads, 1) moe_route_kernel(const __grid_constant__ MoeArgs a) {
  Smem& sm = smem();
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, b = blockIdx.x, routers = a.plan.router_items;
  pdl_begin();
  if (b < routers) {
    router_item(a, b, lane, warp);
    if (finish(a.ctl + MC_ROUTED, sm) == routers - 1) {
      __threadfence();
      select_experts<false>(a, a.logits, true, lane, warp);
      publish_routing(a, sm);
      if (threadIdx.x == 0) a.ctl[MC_ROUTED] = 0;
    }
  } else {
    const size_t i0 = (size_t)(b - routers) * kMThreads + threadIdx.x;
    split_x(a, i0);
    const size_t step = (size_t)(gridDim.x - routers) * kMThreads;
    const int sb = a.d_model / 32, pitch = moe_xs_pitch(a.d_model), rest = pitch - sb;
    for (size_t i = i0; i < (size_t)a.T * rest; i += step) a.xs[i / rest * pitch + sb + i % rest] = 0;
  }
}

template <bool FP4, bool ONE>
__global__ void __launch_bounds__(kThreads, 1) moe_kernel(const __grid_constant__ MoeArgs a) {
  Smem& sm = smem();
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const bool computes = warp < kMWarps;
  const MoePlan& P = a.plan;
  const Ring R{P.row_bytes, P.scale_bytes, P.stage_bytes, P.pitch, P.stage_rows, P.stages, P.x_bytes};
  RingAt at, atd;
  if (threadIdx.x == 0) {
    for (int i = 0; i < R.stages; ++i) {
      mbar_init(&sm.full[i], 1);
      mbar_init(&sm.empty[i], kMWarps);
    }
    for (int i = 0; i < P.down_stages; ++i) {
      mbar_init(&sm.dfull[i], 1);
      mbar_init(&sm.dempty[i], kMWarps);
    }
    for (int i = 0; i < 4; ++i) {
      mbar_init(&sm.listed[i], kBatch);
      mbar_init(&sm.taken[i], 1);
    }
    mbar_fence_init();
    sm.abort = 0;
  }
  pdl_begin();
  int S = 1, nD = 0;                    // known once the experts are
  bool routed = false;
  if (threadIdx.x == 0) sm.item = atomicAdd(a.ctl + MC_QUEUE, 1);
  __syncthreads();
  for (;;) {
    const int item = sm.item;
    __syncthreads();
    int i = item;
    if (i < P.router_items) {
      if (computes) {
        if (i < P.router_items - P.x_items) {
          router_item(a, i, lane, warp);
        } else {
          const int t = (i - (P.router_items - P.x_items)) * kMWarps + warp;
          if (t < a.T) {
            const float u = x_power(a.x + (size_t)t * a.d_model, a.d_model, lane);
            if (lane == 0) __stcg(a.xup + t, u);
          }
        }
        if (finish(a.ctl + MC_ROUTED, sm) == P.router_items - 1) {
          __threadfence();
          select_experts<false>(a, a.logits, true, lane, warp);
          publish_routing(a, sm);
          finish(a.ctl + MC_READY, sm);
        }
      }
    } else {
      i -= P.router_items;
      if (!routed) {
        if (computes) {
          if (P.local) {
            route_here(a, item == 0, lane, warp);
          } else if (wait_for(a.ctl + MC_READY, 1, a.status, 70, sm)) {
            fetch_routing(a, sm);
          } else if (threadIdx.x == 0) {
            sm.active = 0;              // no tables to go by
          }
          csync();
          count_passes(a, sm);
        }
        __syncthreads();
        if (sm.active == 0) break;
        routed = true;
        if constexpr (!ONE) {
          S = down_splits(a, sm);
          nD = down_items(a, sm, S);
        }
      }
      if (i < P.hidden_items) {
        hidden_item<FP4, ONE>(a, R, at, sm, i, lane, warp);
        if (computes) finish(a.ctl + MC_HIDDEN, sm);
      } else if ((i -= P.hidden_items) < nD) {
        if constexpr (!ONE) {
          if (computes) wait_for(a.ctl + MC_HIDDEN, P.hidden_items, a.status, 71, sm);
          // (the copying warp waits for the first list of rows)
          down_item(a, atd, sm, i, S, lane, warp);
          if (computes) finish(a.ctl + MC_DOWN, sm);
        }
      } else if ((i -= nD) < P.out_items) {
        if (computes) {
          if (ONE) wait_for(a.ctl + MC_HIDDEN, P.hidden_items, a.status, 72, sm);
          else wait_for(a.ctl + MC_DOWN, nD, a.status, 73, sm);
          sum_item(a, sm, i, S);
        }
      } else {
        break;
      }
    }
    // (drawn when the item is done: a CTA that holds its next item beforehand
    // takes two of the hidden layer's equal shares while another takes none)
    if (threadIdx.x == 0) sm.item = atomicAdd(a.ctl + MC_QUEUE, 1);
    __syncthreads();
  }
  // after a wait that gave up, copies may still be in flight
  if (warp == kMWarps && lane == 0 && *(volatile int*)&sm.abort) {
    for (int k = 1; k <= R.stages && k <= at.issued; ++k) {
      const int g = at.issued - k;
      mbar_wait(&sm.full[g % R.stages], (uint32_t)(g / R.stages) & 1u);
    }
    for (int k = 1; k <= P.down_stages && k <= atd.issued; ++k) {
      const int g = atd.issued - k;
      mbar_wait(&sm.dfull[g % P.down_stages], (uint32_t)(g / P.down_stages) & 1u);
    }
  }
  // the last CTA to leave clears the counters for the next call
  if (threadIdx.x == 0) {
    __threadfence();
    if (atomicAdd(a.ctl + MC_EXIT, 1) == (int)gridDim.x - 1)
      for (int c = 0; c < MC_COUNT; ++c) a.ctl[c] = 0;
  }
}

// One kernel or the tensor-core ones.
// 4-bit weights: one token's layer (d_model <= 4096) in this kernel, everything else
// by the tensor-core kernels, which read all weights but expand none of them in
// registers.  One token, this kernel / the tensor-core ones, us, dReLU (79% of the gates closed;
// squared ReLU): 2 of 8 experts of 11008 x 4096 53 / 74 (74 / 74), 4 of 60 of 1408 x 2048 32 / 41
// (37 / 41), 2 of 16 of 512 x 512 22 / 30 (23 / 29).  (Several tokens in registers: 8 tokens of the
// first layer 244, 64 tokens 1089, on the tensor cores 190 and 271.)
// bf16 weights: reading every row costs no more than picking the open ones once two
// tokens share an expert, or where an expert's rows take less time than the batches'
// waits.  The same layers: first 2 tokens 138 / 151 (186 / 151), 4: 232 / 287 (322 / 285), 8: 308 /
// 316 (418 / 317), 64: 878 / 371 (994 / 372); second 2 tokens 59 / 55 (64 / 53), 8: 104 / 105 (132 / 105),
// 64: 370 / 251 (418 / 250); third 4 tokens 34 / 28 (35 / 27).  Sizes do not tell how often gates are
// closed: the first layer's 8 tokens (8 experts used) take 441 / 345 with 50% of them closed, 276 / 345 with
// 93%, 239 / 345 with 99%; the rule is made for what is closed about as often as in the cases.
// f32 results: matrix instructions cut a sum off at each step, 3e-8 of it.  This kernel's
// sums over d_model and its down sums (200 steps and more) put y off by 2e-6 to 3e-6, the bf16
// tensor-core kernels' (which add up every 128 terms) by 6e-7: those for every call of several
// tokens or of d_model above 4096 (one token, whose results are bf16 or whose d_model is at most
// 4096, stays here: 2 of 4 experts of 11008 x 8192, f32: 330 / 210 us, of 64 of 1024 x 8192: 69 / 78).  4-bit
// weights: sums of 1024 neurons (4e-7, as of a plain float32 product), of 2048 for bf16 results
// (8e-7; 32 tokens of the first layer 204 instead of 216 us).
MoePlan make_plan(int T, int d_model, int d_ff, int n_experts, int top_k, bool y_bf16) {
  constexpr bool fp4 = kFp4;
  MoePlan p;
  p.grid = kNumSMs;
  p.one_token = T == 1 && d_model <= 4096;
  const long used = n_experts < T * top_k ? n_experts : T * top_k;
  p.tensor = fp4 ? !p.one_token
                 : !p.one_token &&
                       (!y_bf16 || (T > 1 && (T * top_k >= 2 * n_experts || used * d_ff * d_model * 6 < (256l << 20))));
  p.local = !p.tensor && T <= 8 && n_experts <= 64 && n_experts * d_model <= 65536;
  p.x_items = !p.local && fp4 && !p.tensor;
  p.router_items = p.local ? 0 : (n_experts + 15) / 16 * ((T + 7) / 8) + p.x_items;
  p.hidden_items = p.grid;
  // tokens per pass: two groups of 8 where x of both fits the registers; 4-bit
  // weights: the one token, x in shared memory
  p.hidden_tokens = fp4 ? 1 : d_model <= 4096 ? 16 : 8;
  p.x_bytes = fp4 ? (d_model * 2 + 127) / 128 * 128 : 0;
  // the ring: stages of about 36 KB, whole tiles of 8 or 16 rows where rows are
  // short
  p.row_bytes = fp4 ? d_model / 2 : d_model * 2;
  // eight rows' loads of 64 or 16 bytes each do not meet in a bank
  const int apart = fp4 ? 16 : 64, tile = fp4 ? 16 : 8;
  p.scale_bytes = fp4 && d_model % 512 == 0 ? d_model / 32 : 0;     // what bulk copies can take
  p.pitch = (p.row_bytes + 127 - apart) / 128 * 128 + apart;
  p.stage_rows = 36 * 1024 / (p.pitch + p.scale_bytes);
  if (p.stage_rows < 1) p.stage_rows = 1;
  if (p.stage_rows > tile) p.stage_rows = p.stage_rows > 64 ? 64 : p.stage_rows / tile * tile;
  p.stage_bytes = (p.stage_rows * (p.pitch + p.scale_bytes) + 127) / 128 * 128;
  p.stages = (kTail - p.x_bytes) / p.stage_bytes;
  if (p.stages > kMaxStages) p.stages = kMaxStages;
  if (p.tensor) {
    p.down_tokens = kMoeDownTokens;
    p.tile_cols = fp4 ? kMoeDownCols : kMoeDownColsBf16;
    p.col_tiles = (d_model + p.tile_cols - 1) / p.tile_cols;
  } else {
    // the down projection: tiles of the warps' strips
    p.down_tokens = T <= 8 ? 8 : 16;
    p.tile_cols = kMWarps * (p.down_tokens == 8 ? kStrips : kStrips / 2) * 64;
    if (p.tile_cols > d_model) p.tile_cols = d_model;
    p.col_tiles = (d_model + p.tile_cols - 1) / p.tile_cols;
    // 32 mod 128: four rows' loads do not meet in a bank
    p.down_pitch = (p.tile_cols * 2 + 95) / 128 * 128 + 32;
    p.down_stages = kTail / (kRowsStage * p.down_pitch);
    if (p.down_stages > kMaxStages) p.down_stages = kMaxStages;
  }
  const long vecs = ((long)T * (d_model / 4) + 15) / 16;
  p.out_items = (int)(vecs < p.grid ? vecs : p.grid);
  p.max_splits = kMoePartRows / (T * top_k);
  if (p.max_splits < 1) p.max_splits = 1;
  if (p.max_splits > p.grid) p.max_splits = p.grid;
  // (tensor cores: at least four steps of 64 neurons)
  if (p.tensor && p.max_splits > d_ff / 256) p.max_splits = d_ff < 512 ? 1 : d_ff / 256;
  p.sum_steps = y_bf16 ? 32 : 16;
  return p;
}

cudaError_t launch(const MoeArgs& a, cudaStream_t s) {
  cudaError_t e;
  if (a.plan.tensor) {
    static unsigned done = 0;
    e = ensure_smem_attr(moe_route_kernel, (int)sizeof(Smem), &done);
    if (e != cudaSuccess) return e;
    const size_t splits = kFp4 ? ((size_t)a.T * a.d_model / 8 + kMThreads - 1) / kMThreads : 0;
    e = launch_pdl(moe_route_kernel, dim3((unsigned)(a.plan.router_items + splits)), dim3(kMThreads), sizeof(Smem), s, a);
    if constexpr (kFp4) {
      if (e == cudaSuccess) e = launch_moe_fp4_factors(a, s);
      if (e == cudaSuccess) e = launch_moe_fp4_down(a, s);
    } else {
      if (e == cudaSuccess) e = launch_moe_bf16_tensor(a, s);
    }
    if (e == cudaSuccess) e = launch_moe_sum(a, s);
    return e != cudaSuccess ? e : cudaGetLastError();
  }
  auto run = [&](auto kernel, unsigned* done) {
    const cudaError_t r = ensure_smem_attr(kernel, (int)sizeof(Smem), done);
    if (r != cudaSuccess) return r;
    return launch_pdl(kernel, dim3((unsigned)a.plan.grid), dim3(kThreads), sizeof(Smem), s, a);
  };
  static unsigned done_one = 0;
  if constexpr (kFp4) {
    e = run(moe_kernel<true, true>, &done_one);
  } else {
    static unsigned done_many = 0;
    e = a.plan.one_token ? run(moe_kernel<false, true>, &done_one) : run(moe_kernel<false, false>, &done_many);
  }
  if (e != cudaSuccess) return e;
  return cudaGetLastError();
}

}  // namespace
}  // namespace qs
