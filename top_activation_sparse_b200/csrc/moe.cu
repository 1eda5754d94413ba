// A whole mixture-of-experts FFN layer for up to 64 tokens in one kernel.
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
//   router  logits of 8 experts x 8 tokens per item; the CTA that finishes the
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
// Products run on mma.sync m16n8k16 (16 neurons x 8 tokens, or 16 columns x 8
// tokens): with weights read once, up to 64 tokens stay bound by bytes, and
// the operands go from global memory to registers without shared memory (the
// sum over k may be permuted freely as long as both operands agree; a lane's
// 16 bytes are its k values).  x and bf16 weights enter exactly; h enters as
// the sum of three bf16 numbers (relative error below 2^-24).  4-bit weights are
// expanded in registers to bf16, exactly.
#include "moe.cuh"

namespace qs {
namespace {

constexpr int kMThreads = 256;
constexpr int kMWarps = kMThreads / 32;
constexpr int kMaxNg = 4;              // groups of 8 tokens per pass
constexpr int kRowsA = 128;            // neurons per round of the hidden layer
constexpr int kListD = 2048;           // neurons per round of the down projection
constexpr int kRowsD = 128;            // flagged neurons whose h is staged at a time
constexpr int kHPitch = kRowsD + 16;   // bf16 entries per token (pitch = 32 bytes mod 128)

struct Smem {
  union {
    struct {
      float red[kMWarps * 32 * 8 * kMaxNg];      // 32 KB: the warps' partial sums of a 32-neuron tile
      float first[kRowsA * 8 * kMaxNg];          // 16 KB: first factors
      int rows[kRowsA];                          // neurons of the current pass (-1: none)
      uint8_t flag[kRowsA];
    } a;
    struct {
      __nv_bfloat16 h[3][8 * kMaxNg * kHPitch];
      uint16_t list[kListD];
    } d;
    struct {
      int sel[kMoeMaxSlots];
    } r;
  };
  int tok[8 * kMaxNg];                           // the pass's tokens (-1: none)
  int scan[kMWarps];
  int item, count, last;
};

__device__ __forceinline__ uint4 ld_w(const uint8_t* p) {
  uint4 r;
  asm volatile("ld.global.nc.L1::no_allocate.L2::256B.v4.u32 {%0,%1,%2,%3}, [%4];"
               : "=r"(r.x), "=r"(r.y), "=r"(r.z), "=r"(r.w)
               : "l"(p));
  return r;
}
__device__ __forceinline__ uint2 ld_w8(const uint8_t* p) {
  uint2 r;
  asm volatile("ld.global.nc.L1::no_allocate.L2::256B.v2.u32 {%0,%1}, [%2];" : "=r"(r.x), "=r"(r.y) : "l"(p));
  return r;
}
__device__ __forceinline__ uint4 ld_x(const __nv_bfloat16* p) {
  uint4 r;
  asm volatile("ld.global.nc.v4.u32 {%0,%1,%2,%3}, [%4];" : "=r"(r.x), "=r"(r.y), "=r"(r.z), "=r"(r.w) : "l"(p));
  return r;
}

__device__ __forceinline__ void mma_bf16(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                         uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

__device__ __forceinline__ uint32_t mul_bf16x2(uint32_t a, uint32_t b) {
  uint32_t r;
  asm("mul.rn.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
  return r;
}

// ---- 4-bit weights as bf16 ---------------------------------------------------
// A code's three magnitude bits, put where bf16 has its lowest exponent bits
// and its highest mantissa bit, read as value * 2^-126 (subnormals included);
// one product brings in 2^126 and the block's scale: 2^126 2^(s-127) = 2^(s-1)
// for scales up to 2, a second product the rest of larger ones.
struct Scale2 {
  uint32_t lo, hi;     // factors (bf16 pairs); hi is applied where s > 128
};
__device__ __forceinline__ uint32_t scale_lo(uint32_t s) { return (s < 128u ? s + 126u : 254u) << 7; }
__device__ __forceinline__ uint32_t scale_hi(uint32_t s) { return s == 255u ? 0x7fc0u : (s > 128u ? s - 1u : 127u) << 7; }

// bits 4c..4c+3 of each half of p -> a pair of bf16 magnitudes times 2^-126
template <int C>
__device__ __forceinline__ uint32_t code_pair(uint32_t p) {
  const uint32_t m = C == 0 ? p << 6 : C == 1 ? p << 2 : C == 2 ? p >> 2 : p >> 6;
  const uint32_t s = C == 3 ? p : p << (12 - 4 * C);
  return (m & 0x01c001c0u) | (s & 0x80008000u);
}
template <int C>
__device__ __forceinline__ uint32_t weight_pair(uint32_t p, uint32_t lo, uint32_t hi, bool big) {
  uint32_t v = mul_bf16x2(code_pair<C>(p), lo);
  if (big) v = mul_bf16x2(v, hi);
  return v;
}

// ---- queue and waits ---------------------------------------------------------
__device__ __forceinline__ int ld_acquire(const int32_t* p) {
  int v;
  asm volatile("ld.acquire.gpu.global.s32 %0, [%1];" : "=r"(v) : "l"(p) : "memory");
  return v;
}

// thread 0 waits until *p >= n; everyone leaves together
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
  __syncthreads();
  return sm.last != 0;
}

// the CTA's writes are visible before the count goes up; the count before, to all
__device__ __forceinline__ int finish(int32_t* p, Smem& sm) {
  __threadfence();
  __syncthreads();
  if (threadIdx.x == 0) sm.last = atomicAdd(p, 1);
  __syncthreads();
  return sm.last;
}

// ---- router ------------------------------------------------------------------
// item: 8 experts (one per warp) x 8 tokens
__device__ void router_item(const MoeArgs& a, int item, int lane, int warp) {
  const int ngr = (a.T + 7) / 8;
  const int e = (item / ngr) * kMWarps + warp, t0 = (item % ngr) * 8;
  if (e >= a.E) return;
  const int nt = min(8, a.T - t0);
  const __nv_bfloat16* w = a.router + (size_t)e * a.d_model;
  float s[8];
#pragma unroll
  for (int t = 0; t < 8; ++t) s[t] = 0.0f;
#pragma unroll 4
  for (int k = lane * 8; k < a.d_model; k += 256) {
    const uint4 wv = ld_x(w + k);
    const uint32_t ww[4] = {wv.x, wv.y, wv.z, wv.w};
#pragma unroll
    for (int t = 0; t < 8; ++t) {
      if (t < nt) {
        const uint4 xv = ld_x(a.x + (size_t)(t0 + t) * a.d_model + k);
        const uint32_t xx[4] = {xv.x, xv.y, xv.z, xv.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          s[t] = fmaf(bf16lo(ww[i]), bf16lo(xx[i]), s[t]);
          s[t] = fmaf(bf16hi(ww[i]), bf16hi(xx[i]), s[t]);
        }
      }
    }
  }
#pragma unroll
  for (int t = 0; t < 8; ++t) {
#pragma unroll
    for (int o = 16; o; o >>= 1) s[t] += __shfl_xor_sync(0xffffffffu, s[t], o);
    if (lane == 0 && t < nt) __stcg(a.logits + (size_t)(t0 + t) * a.E + e, s[t]);
  }
}

// larger float, larger key (NaN above all)
__device__ __forceinline__ uint32_t order_key(float f) {
  if (f != f) return 0xffffffffu;
  const uint32_t u = __float_as_uint(f == 0.0f ? 0.0f : f);
  return (u & 0x80000000u) ? ~u : (u | 0x80000000u);
}

// experts and shares of every token, then the experts' token lists
__device__ void select_experts(const MoeArgs& a, Smem& sm, int lane, int warp) {
  const int K = a.top_k;
  for (int t = warp; t < a.T; t += kMWarps) {
    float v[kMoeMaxE / 32];
    uint32_t taken = 0;                       // bit i: this lane's value i is chosen
#pragma unroll
    for (int i = 0; i < kMoeMaxE / 32; ++i) {
      const int e = lane + 32 * i;
      v[i] = e < a.E ? __ldcg(a.logits + (size_t)t * a.E + e) : 0.0f;
    }
    float best = 0.0f, sum = 0.0f, mine = 0.0f;
    int choice = 0;                           // lane j: choice j
    for (int j = 0; j < K; ++j) {
      uint64_t key = 0;                       // order, then the lower expert
#pragma unroll
      for (int i = 0; i < kMoeMaxE / 32; ++i) {
        const int e = lane + 32 * i;
        if (e < a.E && !((taken >> i) & 1u)) {
          const uint64_t k = ((uint64_t)order_key(v[i]) << 32) | (uint32_t)(kMoeMaxE - e);
          key = k > key ? k : key;
        }
      }
#pragma unroll
      for (int o = 16; o; o >>= 1) {
        const uint64_t k = __shfl_xor_sync(0xffffffffu, key, o);
        key = k > key ? k : key;
      }
      const int e = kMoeMaxE - (int)(uint32_t)key;
      float l = 0.0f;
#pragma unroll
      for (int i = 0; i < kMoeMaxE / 32; ++i)
        if (i == (e >> 5)) l = v[i];
      l = __shfl_sync(0xffffffffu, l, e & 31);
      if (lane == (e & 31)) taken |= 1u << (e >> 5);
      if (j == 0) best = l;
      const float p = expf(l - best);
      sum += p;
      if (lane == j) mine = p, choice = e;
    }
    if (lane < K) {
      const float p = mine / sum;
      sm.r.sel[t * K + lane] = choice;
      __stcg(a.share + t * K + lane, p);
      if (a.experts) a.experts[t * K + lane] = choice;
      if (a.weights) a.weights[t * K + lane] = p;
    }
  }
  __syncthreads();
  // thread e: its tokens in order; experts without tokens drop out
  const int n = a.T * K, e = threadIdx.x;
  int cnt = 0;
  if (e < a.E)
    for (int i = 0; i < n; ++i) cnt += sm.r.sel[i] == e;
  const int act = cnt > 0;
  // exclusive sums over the experts: (active experts, slots), both below 2^16
  int v = (act << 16) | cnt, inc = v;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int u = __shfl_up_sync(0xffffffffu, inc, o);
    if (lane >= o) inc += u;
  }
  if (lane == 31) sm.scan[warp] = inc;
  __syncthreads();
  int before = 0, total = 0;
  for (int w = 0; w < kMWarps; ++w) {
    if (w < warp) before += sm.scan[w];
    total += sm.scan[w];
  }
  const int ex = before + inc - v;
  if (act) {
    const int ai = ex >> 16, first = ex & 0xffff;
    __stcg(a.table + kMtExpert + ai, e);
    __stcg(a.table + kMtFirst + ai, first);
    __stcg(a.table + kMtCount + ai, cnt);
    int at = first;
    for (int i = 0; i < n; ++i)
      if (sm.r.sel[i] == e) {
        __stcg(a.table + kMtToken + at, i / K);
        __stcg(a.table + kMtSlot + i, at);
        ++at;
      }
  }
  if (threadIdx.x == 0) __stcg(a.table, total >> 16);
}

// ---- hidden layer ------------------------------------------------------------
// 32 neurons (rows[0..31], -1: none) x 8 NG tokens: the eight warps take every
// eighth piece of 128 bytes of the rows and leave their sums in red
template <bool FP4, int NG>
__device__ __forceinline__ void tile_dot(const uint8_t* w, const uint8_t* sc, const int* rows, const MoeArgs& a,
                                         const int* tok, float* red, int lane, int warp) {
  const int g = lane >> 2, q = lane & 3;
  const size_t rb = FP4 ? (size_t)(a.d_model / 2) : (size_t)a.d_model * 2;     // bytes of a row
  const int sb = a.d_model / 32;
  constexpr int kLane = FP4 ? 32 : 8;                   // values of a lane's 16 bytes
  const uint8_t* p[4];
  const uint8_t* ps[4];
#pragma unroll
  for (int r = 0; r < 4; ++r) {
    const int j = rows[g + 8 * r];
    p[r] = j < 0 ? nullptr : w + (size_t)j * rb;
    ps[r] = (!FP4 || j < 0) ? nullptr : sc + (size_t)j * sb;
  }
  const __nv_bfloat16* px[NG];
#pragma unroll
  for (int n = 0; n < NG; ++n) px[n] = tok[n * 8 + g] < 0 ? nullptr : a.x + (size_t)tok[n * 8 + g] * a.d_model;
  float acc[2][NG][4];
#pragma unroll
  for (int m = 0; m < 2; ++m)
#pragma unroll
    for (int n = 0; n < NG; ++n)
#pragma unroll
      for (int i = 0; i < 4; ++i) acc[m][n][i] = 0.0f;
  const int pieces = (a.d_model + 8 * kLane - 1) / (8 * kLane);     // of 128 bytes: two quads of lanes' 16
  const uint4 zero = make_uint4(0, 0, 0, 0);

  auto load = [&](int pc, uint4 (&wv)[2][4], uint32_t (&s)[2][4]) {
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const int k = pc * 8 * kLane + (h * 4 + q) * kLane;
      const bool in = pc < pieces && k < a.d_model;
#pragma unroll
      for (int r = 0; r < 4; ++r) {
        wv[h][r] = (in && p[r]) ? ld_w(p[r] + (FP4 ? k / 2 : k * 2)) : zero;
        if (FP4) s[h][r] = (in && ps[r]) ? (uint32_t)__ldg(ps[r] + k / 32) : 0u;
      }
    }
  };
  uint4 wv[2][2][4];
  uint32_t s[2][2][4];
  load(warp, wv[0], s[0]);
  for (int pc = warp, b = 0; pc < pieces; pc += 2 * kMWarps) {
#pragma unroll
    for (b = 0; b < 2; ++b) {
      const int pb = pc + b * kMWarps;
      if (pb >= pieces) break;
      load(pb + kMWarps, wv[b ^ 1], s[b ^ 1]);
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const int k = pb * 8 * kLane + (h * 4 + q) * kLane;
        const bool in = k < a.d_model;
        if constexpr (!FP4) {
          const uint32_t* w0 = reinterpret_cast<const uint32_t*>(&wv[b][h][0]);
          const uint32_t* w1 = reinterpret_cast<const uint32_t*>(&wv[b][h][1]);
          const uint32_t* w2 = reinterpret_cast<const uint32_t*>(&wv[b][h][2]);
          const uint32_t* w3 = reinterpret_cast<const uint32_t*>(&wv[b][h][3]);
#pragma unroll
          for (int n = 0; n < NG; ++n) {
            const uint4 xv = (in && px[n]) ? ld_x(px[n] + k) : zero;
            const uint32_t* xw = reinterpret_cast<const uint32_t*>(&xv);
#pragma unroll
            for (int i = 0; i < 4; i += 2) {
              mma_bf16(acc[0][n], w0[i], w1[i], w0[i + 1], w1[i + 1], xw[i], xw[i + 1]);
              mma_bf16(acc[1][n], w2[i], w3[i], w2[i + 1], w3[i + 1], xw[i], xw[i + 1]);
            }
          }
        } else {
          uint32_t lo[4], hi[4];
          bool big[4];
#pragma unroll
          for (int r = 0; r < 4; ++r) {
            lo[r] = scale_lo(s[b][h][r]) * 0x10001u;
            hi[r] = scale_hi(s[b][h][r]) * 0x10001u;
            big[r] = s[b][h][r] > 128u;
          }
#pragma unroll
          for (int i = 0; i < 4; ++i) {                // words of 8 codes
            uint32_t f[4][4];
#pragma unroll
            for (int r = 0; r < 4; ++r) {
              const uint32_t c = reinterpret_cast<const uint32_t*>(&wv[b][h][r])[i];
              f[r][0] = weight_pair<0>(c, lo[r], hi[r], big[r]);     // codes 0, 4
              f[r][1] = weight_pair<1>(c, lo[r], hi[r], big[r]);     // codes 1, 5
              f[r][2] = weight_pair<2>(c, lo[r], hi[r], big[r]);
              f[r][3] = weight_pair<3>(c, lo[r], hi[r], big[r]);
            }
#pragma unroll
            for (int n = 0; n < NG; ++n) {
              const uint4 xv = (in && px[n]) ? ld_x(px[n] + k + 8 * i) : zero;
              const uint32_t b0 = __byte_perm(xv.x, xv.z, 0x5410), b1 = __byte_perm(xv.x, xv.z, 0x7632);
              const uint32_t b2 = __byte_perm(xv.y, xv.w, 0x5410), b3 = __byte_perm(xv.y, xv.w, 0x7632);
              mma_bf16(acc[0][n], f[0][0], f[1][0], f[0][1], f[1][1], b0, b1);
              mma_bf16(acc[1][n], f[2][0], f[3][0], f[2][1], f[3][1], b0, b1);
              mma_bf16(acc[0][n], f[0][2], f[1][2], f[0][3], f[1][3], b2, b3);
              mma_bf16(acc[1][n], f[2][2], f[3][2], f[2][3], f[3][3], b2, b3);
            }
          }
        }
      }
    }
  }
  float* o = red + warp * 32 * 8 * NG;
#pragma unroll
  for (int m = 0; m < 2; ++m)
#pragma unroll
    for (int n = 0; n < NG; ++n) {
      *reinterpret_cast<float2*>(o + (m * 16 + g) * 8 * NG + n * 8 + 2 * q) = make_float2(acc[m][n][0], acc[m][n][1]);
      *reinterpret_cast<float2*>(o + (m * 16 + g + 8) * 8 * NG + n * 8 + 2 * q) = make_float2(acc[m][n][2], acc[m][n][3]);
    }
}

__device__ __forceinline__ float relu_nan(float v) { return v <= 0.0f ? 0.0f : v; }   // keeps a NaN

// neurons [j0, j1) of active expert ai for its tokens t0 .. t0 + nt of the list
template <bool FP4, int NG>
__device__ void hidden_rows(const MoeArgs& a, Smem& sm, int ai, int e, int slot0, int nt, int j0, int j1, bool add,
                            bool keep_zeros, int lane, int warp) {
  const size_t mat = (size_t)a.d_ff * a.d_model;
  const size_t wo = FP4 ? (size_t)e * (mat / 2) : (size_t)e * mat * 2, so = FP4 ? (size_t)e * (mat / 32) : 0;
  const int tid = threadIdx.x;
  const float* b1 = a.b1 ? a.b1 + (size_t)e * a.d_ff : nullptr;
  const float* b2 = a.b2 ? a.b2 + (size_t)e * a.d_ff : nullptr;
  for (int jb = j0; jb < j1; jb += kRowsA) {
    const int nr = min(kRowsA, j1 - jb);
    // first factor of every neuron
    for (int i = tid; i < kRowsA; i += kMThreads) {
      sm.a.rows[i] = i < nr ? jb + i : -1;
      sm.a.flag[i] = 0;
    }
    __syncthreads();
    for (int r0 = 0; r0 < nr; r0 += 32) {
      tile_dot<FP4, NG>(a.w1 + wo, FP4 ? a.s1 + so : nullptr, sm.a.rows + r0, a, sm.tok, sm.a.red, lane, warp);
      __syncthreads();
      for (int i = tid; i < 32 * 8 * NG; i += kMThreads) {
        float v = 0.0f;
#pragma unroll
        for (int w = 0; w < kMWarps; ++w) v += sm.a.red[w * 32 * 8 * NG + i];
        const int r = r0 + i / (8 * NG);
        if (b1 && r < nr) v += b1[jb + r];
        v = relu_nan(v);
        if (!a.drelu) v *= v;
        sm.a.first[r * 8 * NG + i % (8 * NG)] = v;
        if (r < nr && i % (8 * NG) < nt && v != 0.0f) sm.a.flag[r] = 1;
      }
      __syncthreads();
    }
    // the open neurons, in order
    if (warp == 0) {
      int n = 0;
      for (int i = lane; i < kRowsA; i += 32) {
        const bool open = sm.a.flag[i] != 0;
        const unsigned m = __ballot_sync(0xffffffffu, open);
        if (open) sm.a.rows[n + __popc(m & lanemask_lt())] = jb + i;
        n += __popc(m);
      }
      for (int i = n + lane; i < min(kRowsA, (n + 31) & ~31); i += 32) sm.a.rows[i] = -1;
      if (lane == 0) sm.count = n;
    }
    // a closed neuron's h is 0 and is not read again: only its flag is written
    // (unless another pass's tokens may open it)
    for (int i = tid; i < nr; i += kMThreads)
      if (!sm.a.flag[i]) {
        if (!add) a.nz[(size_t)ai * a.d_ff + jb + i] = 0;
        if (keep_zeros)
          for (int c = 0; c < nt; ++c) __stcg(a.h + (size_t)(slot0 + c) * a.d_ff + jb + i, 0.0f);
      }
    __syncthreads();
    const int n = sm.count;
    for (int r0 = 0; r0 < n; r0 += 32) {
      tile_dot<FP4, NG>(a.w2 + wo, FP4 ? a.s2 + so : nullptr, sm.a.rows + r0, a, sm.tok, sm.a.red, lane, warp);
      __syncthreads();
      // one neuron per 8 NG neighbouring threads
      for (int i = tid; i < 32 * 8 * NG; i += kMThreads) {
        const int r = r0 + i / (8 * NG), c = i % (8 * NG);
        float h = 0.0f;
        const int j = r < n ? sm.a.rows[r] : -1;
        if (j >= 0 && c < nt) {
          float v = 0.0f;
#pragma unroll
          for (int w = 0; w < kMWarps; ++w) v += sm.a.red[w * 32 * 8 * NG + i];
          if (b2) v += b2[j];
          if (a.drelu) v = relu_nan(v);
          h = sm.a.first[(j - jb) * 8 * NG + c] * v;
          __stcg(a.h + (size_t)(slot0 + c) * a.d_ff + j, h);
        }
        const unsigned any = __ballot_sync(0xffffffffu, h != 0.0f);
        const unsigned mine = NG == 4 ? any : (any >> ((lane / (8 * NG)) * 8 * NG)) & ((1u << (8 * NG & 31)) - 1u);
        if (j >= 0 && c == 0) {
          uint8_t* f = a.nz + (size_t)ai * a.d_ff + j;
          if (add) { if (mine) *f = 1; }
          else *f = mine != 0;
        }
      }
      __syncthreads();
    }
  }
}

// The tokens of an active expert in passes of up to 32, each with the smallest
// instance that holds it.
template <typename F>
__device__ __forceinline__ void token_passes(const MoeArgs& a, Smem& sm, int first, int cnt, F&& f) {
  for (int t0 = 0; t0 < cnt; t0 += 8 * kMaxNg) {
    const int nt = min(8 * kMaxNg, cnt - t0);
    __syncthreads();
    if (threadIdx.x < 8 * kMaxNg)
      sm.tok[threadIdx.x] = (int)threadIdx.x < nt ? __ldcg(a.table + kMtToken + first + t0 + threadIdx.x) : -1;
    __syncthreads();
    f(t0, nt);
  }
}

template <bool FP4>
__device__ void hidden_item(const MoeArgs& a, Smem& sm, int item, int lane, int warp) {
  const int A = __ldcg(a.table);
  const long long N = (long long)A * a.d_ff;
  long long n0 = N * item / a.plan.hidden_items;
  const long long n1 = N * (item + 1) / a.plan.hidden_items;
  while (n0 < n1) {
    const int ai = (int)(n0 / a.d_ff), j0 = (int)(n0 - (long long)ai * a.d_ff);
    const int j1 = (int)min((long long)a.d_ff, (long long)j0 + (n1 - n0));
    const int e = __ldcg(a.table + kMtExpert + ai), first = __ldcg(a.table + kMtFirst + ai), cnt = __ldcg(a.table + kMtCount + ai);
    token_passes(a, sm, first, cnt, [&](int t0, int nt) {
      if (nt <= 8) hidden_rows<FP4, 1>(a, sm, ai, e, first + t0, nt, j0, j1, t0 > 0, cnt > 8 * kMaxNg, lane, warp);
      else if (nt <= 16) hidden_rows<FP4, 2>(a, sm, ai, e, first + t0, nt, j0, j1, t0 > 0, cnt > 8 * kMaxNg, lane, warp);
      else hidden_rows<FP4, 4>(a, sm, ai, e, first + t0, nt, j0, j1, t0 > 0, cnt > 8 * kMaxNg, lane, warp);
    });
    n0 += j1 - j0;
  }
}

// ---- down projection ---------------------------------------------------------
// a strip of 64 (bf16) or 128 (4-bit) columns per warp; the CTA's flagged
// neurons of [j0, j1) are listed once and their h staged as three bf16 parts
template <bool FP4, int NG>
__device__ void down_rows(const MoeArgs& a, Smem& sm, int ai, int e, int slot0, int nt, int j0, int j1, int strip,
                          int split, int lane, int warp) {
  constexpr int kCols = FP4 ? 16 : 8;                // columns of a lane
  constexpr int kMma = kCols / 2;                    // MMAs per 16 neurons and token group
  const int g = lane >> 2, q = lane & 3, tid = threadIdx.x;
  const int col = strip * (8 * kCols) + g * kCols;
  // the matrix instructions need whole warps: a strip takes part when its first
  // column exists, a lane loads and stores when its own do (d_model is a
  // multiple of 32, a lane's columns divide that)
  const bool works = strip >= 0 && strip * (8 * kCols) < a.d_model;
  const bool in = works && col < a.d_model;
  const size_t rb = FP4 ? (size_t)(a.d_model / 2) : (size_t)a.d_model * 2;
  const int sb = a.d_model / 32;
  const uint8_t* w = a.wd + (size_t)e * a.d_ff * rb + (FP4 ? col / 2 : col * 2);
  const uint8_t* sc = FP4 ? a.sd + (size_t)e * a.d_ff * sb + col / 32 : nullptr;
  float acc[kMma][NG][4];
#pragma unroll
  for (int m = 0; m < kMma; ++m)
#pragma unroll
    for (int n = 0; n < NG; ++n)
#pragma unroll
      for (int i = 0; i < 4; ++i) acc[m][n][i] = 0.0f;

  for (int jl = j0; jl < j1; jl += kListD) {
    // list the flagged neurons of [jl, je), in order
    const int je = min(j1, jl + kListD);
    int total = 0;
    __syncthreads();
    for (int jb = jl; jb < je; jb += kMThreads) {
      const int j = jb + tid;
      const bool f = j < je && __ldcg(a.nz + (size_t)ai * a.d_ff + j) != 0;
      const unsigned m = __ballot_sync(0xffffffffu, f);
      if (lane == 0) sm.scan[warp] = __popc(m);
      __syncthreads();
      int at = total, sum = 0;
#pragma unroll
      for (int v = 0; v < kMWarps; ++v) {
        if (v < warp) at += sm.scan[v];
        sum += sm.scan[v];
      }
      if (f) sm.d.list[at + __popc(m & lanemask_lt())] = (uint16_t)(j - jl);
      total += sum;
      __syncthreads();
    }
    for (int l0 = 0; l0 < total; l0 += kRowsD) {
      const int n = min(kRowsD, total - l0), np = (n + 15) & ~15;
      // h of these neurons as three bf16 numbers
      for (int i = tid; i < np * 8 * NG; i += kMThreads) {
        const int r = i % np, c = i / np;
        float h = 0.0f;
        if (r < n && c < nt) h = __ldcg(a.h + (size_t)(slot0 + c) * a.d_ff + jl + sm.d.list[l0 + r]);
        // (an infinity or a NaN has no rest)
        const bool finite = fabsf(h) <= 3.0e38f;
#pragma unroll
        for (int v = 0; v < 3; ++v) {
          const __nv_bfloat16 b = __float2bfloat16_rn(h);
          sm.d.h[v][c * kHPitch + r] = b;
          h = finite ? h - __bfloat162float(b) : 0.0f;
        }
      }
      __syncthreads();
      if (works) {
        using Vec = typename std::conditional<FP4, uint2, uint4>::type;
        auto load = [&](int st, Vec (&v)[4], uint32_t (&s)[4]) {
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const int r = st * 16 + 4 * q + i;
            const bool ok = in && r < n;
            const size_t j = ok ? (size_t)(jl + sm.d.list[l0 + r]) : 0;
            if constexpr (FP4) {
              v[i] = ok ? ld_w8(w + j * rb) : make_uint2(0, 0);
              s[i] = ok ? (uint32_t)__ldg(sc + j * sb) : 0u;
            } else {
              v[i] = ok ? ld_w(w + j * rb) : make_uint4(0, 0, 0, 0);
            }
          }
        };
        auto step = [&](int st, const Vec (&v)[4], const uint32_t (&s)[4]) {
          uint2 b[NG][3];
#pragma unroll
          for (int t = 0; t < NG; ++t)
#pragma unroll
            for (int v = 0; v < 3; ++v)
              b[t][v] = *reinterpret_cast<const uint2*>(sm.d.h[v] + (t * 8 + g) * kHPitch + st * 16 + 4 * q);
          auto mmas = [&](int m, uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3) {
#pragma unroll
            for (int t = 0; t < NG; ++t) {
#pragma unroll
              for (int v = 0; v < 3; ++v) mma_bf16(acc[m][t], a0, a1, a2, a3, b[t][v].x, b[t][v].y);
            }
          };
          if constexpr (!FP4) {
            const uint32_t* u0 = reinterpret_cast<const uint32_t*>(&v[0]);
            const uint32_t* u1 = reinterpret_cast<const uint32_t*>(&v[1]);
            const uint32_t* u2 = reinterpret_cast<const uint32_t*>(&v[2]);
            const uint32_t* u3 = reinterpret_cast<const uint32_t*>(&v[3]);
#pragma unroll
            for (int m = 0; m < kMma; ++m)
              mmas(m, __byte_perm(u0[m], u1[m], 0x5410), __byte_perm(u0[m], u1[m], 0x7632),
                   __byte_perm(u2[m], u3[m], 0x5410), __byte_perm(u2[m], u3[m], 0x7632));
          } else {
            // pairs of neurons (0, 1) and (2, 3), one code of each per half
            const uint32_t lo01 = scale_lo(s[0]) | (scale_lo(s[1]) << 16), lo23 = scale_lo(s[2]) | (scale_lo(s[3]) << 16);
            const uint32_t hi01 = scale_hi(s[0]) | (scale_hi(s[1]) << 16), hi23 = scale_hi(s[2]) | (scale_hi(s[3]) << 16);
            const bool b01 = s[0] > 128u || s[1] > 128u, b23 = s[2] > 128u || s[3] > 128u;
#pragma unroll
            for (int half = 0; half < 4; ++half) {     // four columns each
              const uint32_t sel = (half & 1) ? 0x7632 : 0x5410;
              const uint32_t p01 = half < 2 ? __byte_perm(v[0].x, v[1].x, sel) : __byte_perm(v[0].y, v[1].y, sel);
              const uint32_t p23 = half < 2 ? __byte_perm(v[2].x, v[3].x, sel) : __byte_perm(v[2].y, v[3].y, sel);
              mmas(2 * half, weight_pair<0>(p01, lo01, hi01, b01), weight_pair<1>(p01, lo01, hi01, b01),
                   weight_pair<0>(p23, lo23, hi23, b23), weight_pair<1>(p23, lo23, hi23, b23));
              mmas(2 * half + 1, weight_pair<2>(p01, lo01, hi01, b01), weight_pair<3>(p01, lo01, hi01, b01),
                   weight_pair<2>(p23, lo23, hi23, b23), weight_pair<3>(p23, lo23, hi23, b23));
            }
          }
        };
        const int nst = np / 16;
        Vec v0[4], v1[4], v2[4];
        uint32_t s0[4], s1[4], s2[4];
        load(0, v0, s0);
        load(1, v1, s1);
        for (int st = 0; st < nst; st += 3) {          // two steps ahead
          load(st + 2, v2, s2);
          step(st, v0, s0);
          if (st + 1 >= nst) break;
          load(st + 3, v0, s0);
          step(st + 1, v1, s1);
          if (st + 2 >= nst) break;
          load(st + 4, v1, s1);
          step(st + 2, v2, s2);
        }
      }
      __syncthreads();
    }
  }
  if (in) {
    const size_t slots = (size_t)a.T * a.top_k;
#pragma unroll
    for (int t = 0; t < NG; ++t)
#pragma unroll
      for (int c = 0; c < 2; ++c) {
        const int n = t * 8 + 2 * q + c;
        if (n < nt) {
          float* o = a.parts + ((size_t)split * slots + slot0 + n) * a.d_model + col;
#pragma unroll
          for (int m = 0; m < kMma; m += 2)
            __stcg(reinterpret_cast<float4*>(o + 2 * m),
                   make_float4(acc[m][t][c], acc[m][t][2 + c], acc[m + 1][t][c], acc[m + 1][t][2 + c]));
        }
      }
  }
}

// splits of an expert's neurons: about one item per CTA in all
__device__ __forceinline__ int down_splits(const MoeArgs& a, int A) {
  const int s = a.plan.grid / (A * a.plan.col_tiles);
  return max(1, min(s, a.plan.max_splits));
}

template <bool FP4>
__device__ void down_item(const MoeArgs& a, Smem& sm, int item, int A, int S, int lane, int warp) {
  const int ct = item % a.plan.col_tiles, rest = item / a.plan.col_tiles, s = rest % S, ai = rest / S;
  const int e = __ldcg(a.table + kMtExpert + ai), first = __ldcg(a.table + kMtFirst + ai), cnt = __ldcg(a.table + kMtCount + ai);
  const int j0 = (int)((long long)a.d_ff * s / S), j1 = (int)((long long)a.d_ff * (s + 1) / S);
  const int strip = warp < a.plan.tile_warps ? ct * a.plan.tile_warps + warp : -1;
  token_passes(a, sm, first, cnt, [&](int t0, int nt) {
    // the 4-bit form has twice the columns, and half the tokens, per warp
    if (nt <= 8) down_rows<FP4, 1>(a, sm, ai, e, first + t0, nt, j0, j1, strip, s, lane, warp);
    else if (nt <= 16) down_rows<FP4, 2>(a, sm, ai, e, first + t0, nt, j0, j1, strip, s, lane, warp);
    else if constexpr (!FP4) down_rows<FP4, 4>(a, sm, ai, e, first + t0, nt, j0, j1, strip, s, lane, warp);
    else {
      down_rows<FP4, 2>(a, sm, ai, e, first + t0, 16, j0, j1, strip, s, lane, warp);
      down_rows<FP4, 2>(a, sm, ai, e, first + t0 + 16, nt - 16, j0, j1, strip, s, lane, warp);
    }
  });
}

// ---- sums ----------------------------------------------------------------------
__device__ void sum_item(const MoeArgs& a, int item, int S) {
  const int n4 = a.d_model / 4;
  const long long i = (long long)item * kMThreads + threadIdx.x;
  if (i >= (long long)a.T * n4) return;
  const int t = (int)(i / n4), c = (int)(i - (long long)t * n4) * 4;
  const size_t slots = (size_t)a.T * a.top_k;
  float4 y = make_float4(0, 0, 0, 0);
  for (int j = 0; j < a.top_k; ++j) {
    const int slot = __ldcg(a.table + kMtSlot + t * a.top_k + j);
    const float p = __ldcg(a.share + t * a.top_k + j);
    const float* src = a.parts + (size_t)slot * a.d_model + c;
    float4 v = make_float4(0, 0, 0, 0);
#pragma unroll 8
    for (int s = 0; s < S; ++s) {
      const float4 u = __ldcg(reinterpret_cast<const float4*>(src + (size_t)s * slots * a.d_model));
      v.x += u.x, v.y += u.y, v.z += u.z, v.w += u.w;
    }
    y.x = fmaf(p, v.x, y.x), y.y = fmaf(p, v.y, y.y), y.z = fmaf(p, v.z, y.z), y.w = fmaf(p, v.w, y.w);
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

template <bool FP4>
__global__ void __launch_bounds__(kMThreads, 2) moe_kernel(MoeArgs a) {
  extern __shared__ __align__(16) unsigned char smem_raw[];
  Smem& sm = *reinterpret_cast<Smem*>(smem_raw);
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  pdl_begin();
  const MoePlan& P = a.plan;
  int A = 0, S = 1, nD = 0;             // known once the experts are selected
  if (threadIdx.x == 0) sm.item = atomicAdd(a.ctl + MC_QUEUE, 1);
  __syncthreads();
  for (;;) {
    const int item = sm.item;
    __syncthreads();
    int next = 0;
    if (threadIdx.x == 0) next = atomicAdd(a.ctl + MC_QUEUE, 1);   // asked for early, used at the end
    int i = item;
    if (i < P.router_items) {
      router_item(a, i, lane, warp);
      if (finish(a.ctl + MC_ROUTED, sm) == P.router_items - 1) {
        __threadfence();
        select_experts(a, sm, lane, warp);
        finish(a.ctl + MC_READY, sm);
      }
    } else {
      i -= P.router_items;
      if (A == 0) {
        if (!wait_for(a.ctl + MC_READY, 1, a.status, 70, sm)) break;   // no tables to go by
        A = __ldcg(a.table);
        S = down_splits(a, A);
        nD = A * S * P.col_tiles;
      }
      if (i < P.hidden_items) {
        hidden_item<FP4>(a, sm, i, lane, warp);
        finish(a.ctl + MC_HIDDEN, sm);
      } else if ((i -= P.hidden_items) < nD) {
        wait_for(a.ctl + MC_HIDDEN, P.hidden_items, a.status, 71, sm);
        down_item<FP4>(a, sm, i, A, S, lane, warp);
        finish(a.ctl + MC_DOWN, sm);
      } else if ((i -= nD) < P.out_items) {
        wait_for(a.ctl + MC_DOWN, nD, a.status, 72, sm);
        sum_item(a, i, S);
      } else {
        break;
      }
    }
    if (threadIdx.x == 0) sm.item = next;
    __syncthreads();
  }
  // the last CTA to leave clears the counters for the next call
  if (threadIdx.x == 0) {
    __threadfence();
    if (atomicAdd(a.ctl + MC_EXIT, 1) == (int)gridDim.x - 1)
      for (int c = 0; c < MC_COUNT; ++c) a.ctl[c] = 0;
  }
}

}  // namespace

MoePlan plan_moe(int T, int d_model, int d_ff, int n_experts, int top_k, int fp4) {
  (void)d_ff;
  MoePlan p;
  p.grid = 2 * kNumSMs;
  p.router_items = (n_experts + kMWarps - 1) / kMWarps * ((T + 7) / 8);
  p.hidden_items = p.grid;
  const int strips = (d_model + (fp4 ? 127 : 63)) / (fp4 ? 128 : 64);
  p.col_tiles = (strips + kMWarps - 1) / kMWarps;
  p.tile_warps = (strips + p.col_tiles - 1) / p.col_tiles;
  p.out_items = (int)(((long long)T * (d_model / 4) + kMThreads - 1) / kMThreads);
  p.max_splits = kMoePartRows / (T * top_k);
  if (p.max_splits < 1) p.max_splits = 1;
  if (p.max_splits > p.grid) p.max_splits = p.grid;
  return p;
}

cudaError_t launch_moe(const MoeArgs& a, cudaStream_t s) {
  static unsigned done[2] = {0, 0};
  auto k = a.fp4 ? moe_kernel<true> : moe_kernel<false>;
  cudaError_t e = ensure_smem_attr(k, (int)sizeof(Smem), &done[a.fp4 ? 1 : 0]);
  if (e != cudaSuccess) return e;
  e = launch_pdl(k, dim3((unsigned)a.plan.grid), dim3(kMThreads), sizeof(Smem), s, a);
  if (e != cudaSuccess) return e;
  return cudaGetLastError();
}

}  // namespace qs
