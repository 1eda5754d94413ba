// Both factors of 4-bit experts, and h, on the tensor cores.
//
//   v[t, j] = sum_b s[j, b] sum_{i in block b} q[j, i] x[t, i]
//
// for every neuron j of an expert and its tokens t.  The block-scaled 4-bit
// MMA expands and scales the weights by itself, if x is 4-bit too: x is written
// as a sum of 8 microscaled 4-bit numbers,
//   r_0 = x;  q_i = e2m1(r_i / s_i);  r_{i+1} = r_i - q_i s_i (exact);
//   s_0 = 2^(floor(log2 amax) - 1), s_{i+1} = s_i / 8
// (per block of 32; |r_i / s_i| <= 4, where e2m1's steps are at most 1, so that
// |r_{i+1}| <= s_i / 2: three bits a term).  The rest after 8 terms is at most
// s_7 / 2 = 2^-23 2^floor(log2 amax); a bf16 number not below 2^-15 amax has no rest.
// A token takes 8 columns of the product, whose sums are added in float32, smallest
// first.
//
// Bound by the weights' bytes: 128 neurons x 256 inputs are 16 KB, a token's
// eight columns of the same inputs 1 KB.  32 tokens, 2 of 8 experts of 11008 x 4096
// each: 78 us, 4.9 TB/s of the two matrices' 383 MB.  (Expanding the codes in registers
// for mma.sync took 290 us, ten times the copies.)  Both matrices are read whole: with
// several tokens per expert few neurons are closed for all of them.
//   * warp 0 copies steps of 256 inputs into a ring: 128 rows of both matrices and
//     the 8 rows of each of the pass's tokens (2-D TMA, 128-byte swizzle);
//   * warps 6 to 9 bring the scales of 1024 inputs at a time into the form that
//     tensor memory takes (the weights' lie row by row, a token's 8 columns
//     have one row of scales, three less per term);
//   * one lane of warp 1 copies a step's scales to tensor memory and issues
//     its MMAs (N = 8 columns per token: tokens that a pass does not have cost
//     nothing);
//   * warps 2 to 5 add the terms, form h and store it as three bf16 numbers.
// Units of work (an expert, 128 of its neurons, up to 16 of its tokens) are dealt
// out in turn; the passes of one tile are neighbours, so that the later ones
// find the rows in L2.  Every wait is bounded.
#include "fp4_mma.cuh"
#include "moe_tables.cuh"

namespace qs {
namespace {

constexpr int kFM = 128;                        // neurons per unit
constexpr int kFABytes = kFM * kGK / 2;
constexpr int kFThreads = 320;
constexpr int kMats = 2;                        // matrices: the first factor's, the second's
constexpr int kFTokens = 16;                    // tokens per pass
constexpr int kChunk = 4;                       // steps whose scales come at once
constexpr int kSfOp = kChunk * 2 * kSfTile;     // their bytes per operand
constexpr int kSfRing = 3;
constexpr int kFMaxStages = 8;
constexpr int kFSmemCap = 216 * 1024;

struct FArgs {
  MoeArgs m;
  const uint8_t* xs;                            // [T, xs_pitch] scale bytes of the first terms
  int xs_pitch;
  int tokens;                                   // most tokens of a pass
  int stages, stage_bytes;
  int acc, nacc;                                // accumulator columns per matrix, accumulators
};

struct FUnit {
  int ai, e, m, slot0, nt, np;
};

__device__ __forceinline__ FUnit f_unit(const MoeTables& t, int u, int mtiles) {
  int ai = 0;
  for (int step = kMoeMaxE / 2; step; step >>= 1)
    if (ai + step < t.active && t.cum[ai + step] * mtiles <= u) ai += step;
  FUnit f;
  const int rest = u - t.cum[ai] * mtiles;
  f.np = t.cum[ai + 1] - t.cum[ai];
  f.ai = ai;
  f.e = t.expert[ai];
  f.m = rest / f.np;
  const int t0 = (rest - f.m * f.np) * kFTokens;
  f.slot0 = t.first[ai] + t0;
  f.nt = min(kFTokens, t.count[ai] - t0);
  return f;
}

__device__ __forceinline__ uint32_t f_idesc(uint32_t sf_id, uint32_t n) {
  return (sf_id << 4) | (1u << 7) | (1u << 10) | ((n >> 3) << 17) | (1u << 23) | ((uint32_t)(kFM >> 4) << 24) | (sf_id << 29);
}

__global__ void __launch_bounds__(kFThreads, 1)
    moe_fp4_factors_kernel(const __grid_constant__ CUtensorMap map_1, const __grid_constant__ CUtensorMap map_2,
                         const __grid_constant__ CUtensorMap map_x, const __grid_constant__ FArgs f) {
  extern __shared__ __align__(1024) unsigned char smem_raw[];
  __shared__ __align__(8) uint64_t s_full[kFMaxStages], s_empty[kFMaxStages];
  __shared__ __align__(8) uint64_t s_sffull[kSfRing], s_sfempty[kSfRing];
  __shared__ __align__(8) uint64_t s_tfull[2], s_tempty[2];
  __shared__ __align__(8) uint64_t s_done;
  __shared__ uint32_t s_tmem;
  __shared__ int s_abort;
  __shared__ MoeTables tb;

  const MoeArgs& a = f.m;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const uint32_t base = (smem_u32(smem_raw) + 1023u) & ~1023u;
  const uint32_t sf0 = base + (uint32_t)(f.stages * f.stage_bytes);       // the ring of scales
  constexpr uint32_t kSfSlot = (kMats + 1) * kSfOp;
  const int nk = (a.d_model + kGK - 1) / kGK, nchunk = (nk + kChunk - 1) / kChunk;
  const int mtiles = (a.d_ff + kFM - 1) / kFM;

  if (tid == 0) {
    for (int i = 0; i < f.stages; ++i) mbar_init(&s_full[i], 1), mbar_init(&s_empty[i], 1);
    for (int i = 0; i < kSfRing; ++i) mbar_init(&s_sffull[i], 128), mbar_init(&s_sfempty[i], 1);
    for (int i = 0; i < 2; ++i) mbar_init(&s_tfull[i], 1), mbar_init(&s_tempty[i], 4);
    mbar_init(&s_done, 1);
    mbar_fence_init();
    s_abort = 0;
  }
  if (warp == 1) {
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_u32(&s_tmem)), "r"(512u)
                 : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
  }
  pdl_begin();
  load_tables(a, tb, kFTokens, kFThreads);
  g_before();
  __syncthreads();
  g_after();
  const uint32_t tmem = s_tmem;
  const int units = tb.cum[tb.active] * mtiles;

  if (warp == 0) {
    if (lane == 0) {
      // ---- copies ----
      int i = 0, sl = 0;
      uint32_t ph = 0;
      bool ok = true;
      for (int u = blockIdx.x; u < units && ok; u += gridDim.x) {
        const FUnit x = f_unit(tb, u, mtiles);
        const int row = x.e * a.d_ff + x.m * kFM;
        for (int ks = 0; ks < nk; ++ks, ++i) {
          if (!(ok = g_wait(&s_empty[sl], ph ^ 1u, &s_abort, a.status, 64))) break;
          const uint32_t st = base + (uint32_t)(sl * f.stage_bytes);
          mbar_arrive_expect_tx(&s_full[sl], (uint32_t)(kMats * kFABytes + x.nt * 1024));
          g_tma(st, &map_1, ks * (kGK / 2), row, &s_full[sl]);
          g_tma(st + kFABytes, &map_2, ks * (kGK / 2), row, &s_full[sl]);
          for (int c = 0; c < x.nt; ++c)
            g_tma(st + kMats * kFABytes + c * 1024, &map_x, ks * (kGK / 2), tb.token[x.slot0 + c] * 8, &s_full[sl]);
          if (++sl == f.stages) sl = 0, ph ^= 1u;
        }
      }
      // after a give-up: let the copies in flight land
      if (*(volatile int*)&s_abort)
        for (int j = 0; j < f.stages && j < i; ++j) {
          const int g = i - 1 - j;
          mbar_wait(&s_full[g % f.stages], (uint32_t)(g / f.stages) & 1u);
        }
    }
  } else if (warp == 1) {
    // ---- scales to tensor memory, MMAs.  (The whole warp goes through the steps, one
    // lane issues: what the instructions take is then uniform and need not be moved there
    // lane by lane) ----
    const bool issues = g_elect();
    int sl = 0, sfsl = 0, piece = 0;
    uint32_t ph = 0, sfph = 0;
    bool ok = true;
    const uint32_t sfcols = tmem + (uint32_t)(f.nacc * kMats * f.acc);
    const uint64_t d0 = g_desc(base, 1024, 2), s0 = g_desc(sf0, 128, 0);
    for (int u = blockIdx.x; u < units && ok; u += gridDim.x, ++piece) {
      const FUnit x = f_unit(tb, u, mtiles);
      const uint32_t id0 = f_idesc(0u, (uint32_t)x.nt * 8u), id1 = f_idesc(2u, (uint32_t)x.nt * 8u);
      const int ab = piece % f.nacc;
      if (piece >= f.nacc && !(ok = g_wait_warp(&s_tempty[ab], (uint32_t)(piece / f.nacc - 1) & 1u, &s_abort, a.status, 65))) break;
      g_after();
      const uint32_t acc = tmem + (uint32_t)(ab * kMats * f.acc);
      for (int ks = 0; ks < nk; ++ks) {
        const int in = ks % kChunk;
        if (in == 0 && !(ok = g_wait_warp(&s_sffull[sfsl], sfph, &s_abort, a.status, 66))) break;
        if (!(ok = g_wait_warp(&s_full[sl], ph, &s_abort, a.status, 67))) break;
        g_after();
        const uint64_t st = d0 + (uint64_t)(sl * (f.stage_bytes / 16));
        const uint64_t sfs = s0 + (uint64_t)(sfsl * (int)(kSfSlot / 16) + in * (2 * kSfTile / 16));
        const uint32_t sfc = sfcols + (uint32_t)(sl * (kMats + 1) * 8);
        const int rest = a.d_model - ks * kGK;
        if (issues) {
#pragma unroll
          for (int o = 0; o <= kMats; ++o)
#pragma unroll
            for (int t = 0; t < 2; ++t) g_cp_sf(sfc + o * 8 + t * 4, sfs + o * (kSfOp / 16) + t * (kSfTile / 16));
#pragma unroll
          for (int kk = 0; kk < kGK / 64; ++kk)
            if (kk * 64 < rest) {
#pragma unroll
              for (int o = 0; o < kMats; ++o)
                g_mma<false>(acc + o * f.acc, st + o * (kFABytes / 16) + kk * 2, st + kMats * (kFABytes / 16) + kk * 2,
                             (kk & 1) ? id1 : id0, sfc + o * 8 + (kk >> 1) * 4, sfc + kMats * 8 + (kk >> 1) * 4, ks > 0 || kk > 0);
            }
          g_commit(&s_empty[sl]);
          if (in == kChunk - 1 || ks == nk - 1) g_commit(&s_sfempty[sfsl]);
        }
        __syncwarp();
        if (in == kChunk - 1 || ks == nk - 1)
          if (++sfsl == kSfRing) sfsl = 0, sfph ^= 1u;
        if (++sl == f.stages) sl = 0, ph ^= 1u;
      }
      if (ok && issues) g_commit(&s_tfull[ab]);
    }
    if (issues) {
      g_commit(&s_done);                    // every MMA issued has completed when this arrives
      mbar_wait(&s_done, 0u);
    }
    __syncwarp();
  } else if (warp < 6) {
    // ---- results ----
    const int q = warp & 3;
    int piece = 0;
    for (int u = blockIdx.x; u < units; u += gridDim.x, ++piece) {
      const FUnit x = f_unit(tb, u, mtiles);
      const int ab = piece % f.nacc, j = x.m * kFM + q * 32 + lane;
      const bool mine = j < a.d_ff;
      const size_t bi = (size_t)x.e * a.d_ff + (mine ? j : 0);
      const float b1 = a.b1 ? __ldg(a.b1 + bi) : 0.0f, b2 = a.b2 ? __ldg(a.b2 + bi) : 0.0f;
      if (!g_wait_warp(&s_tfull[ab], (uint32_t)(piece / f.nacc) & 1u, &s_abort, a.status, 68)) break;
      g_after();
      const uint32_t acc = tmem + ((uint32_t)(q * 32) << 16) + (uint32_t)(ab * kMats * f.acc);
      for (int c = 0; c < x.nt; ++c) {
        uint32_t v[kMats][8];
#pragma unroll
        for (int o = 0; o < kMats; ++o) g_ld8(acc + (uint32_t)(o * f.acc + c * 8), v[o]);
        g_ld_wait();
        float s[kMats];
#pragma unroll
        for (int o = 0; o < kMats; ++o) {
          s[o] = __uint_as_float(v[o][7]);
#pragma unroll
          for (int i = 6; i >= 0; --i) s[o] += __uint_as_float(v[o][i]);
        }
        float h = relu_nan(s[0] + b1);
        if (!a.drelu) h *= h;
        // (a closed first factor is 0 whatever the other is)
        float g = s[1] + b2;
        if (a.drelu) g = relu_nan(g);
        h = h == 0.0f ? 0.0f : h * g;
        // h as the sum of three bf16 numbers, for the down projection (an
        // infinity or a NaN has no rest)
        __nv_bfloat16* o = reinterpret_cast<__nv_bfloat16*>(a.h) + (size_t)(x.slot0 + c) * 3 * a.d_ff + j;
        const bool finite = fabsf(h) <= 3.0e38f;
#pragma unroll
        for (int i = 0; i < 3; ++i) {
          const __nv_bfloat16 b = __float2bfloat16_rn(h);
          if (mine) o[(size_t)i * a.d_ff] = b;
          h = finite ? h - __bfloat162float(b) : 0.0f;
        }
      }
      g_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(&s_tempty[ab]);
    }
  } else {
    // ---- scales, a row of the weights and a column of x per thread ----
    const int r = tid - 192, sb = a.d_model / 32;
    const bool wide = sb % 16 == 0;
    const uint32_t at = (uint32_t)((r & 31) * 16 + (r >> 5) * 4);
    int sfsl = 0;
    uint32_t sfph = 0;
    bool ok = true;
    for (int u = blockIdx.x; u < units && ok; u += gridDim.x) {
      const FUnit x = f_unit(tb, u, mtiles);
      const int j = x.m * kFM + r, c = r >> 3;
      const uint8_t* rows[kMats];
      rows[0] = a.s1 + ((size_t)x.e * a.d_ff + j) * sb;
      rows[1] = a.s2 + ((size_t)x.e * a.d_ff + j) * sb;
      const uint8_t* xs = f.xs + (size_t)(c < x.nt ? tb.token[x.slot0 + c] : 0) * f.xs_pitch;
      const uint32_t less = (uint32_t)(3 * (r & 7)) * 0x01010101u;
      for (int ch = 0; ch < nchunk; ++ch) {
        uint32_t w[kMats + 1][8];
#pragma unroll
        for (int o = 0; o < kMats; ++o)
#pragma unroll
          for (int half = 0; half < 2; ++half) {
            const int b = ch * 32 + half * 16;
            uint4 v = make_uint4(0, 0, 0, 0);
            if (j < a.d_ff && b < sb) {
              if (wide) {
                v = __ldg(reinterpret_cast<const uint4*>(rows[o] + b));
              } else {
                uint32_t z[4] = {0, 0, 0, 0};
#pragma unroll
                for (int i = 0; i < 16; ++i)
                  if (b + i < sb) z[i >> 2] |= (uint32_t)__ldg(rows[o] + b + i) << (8 * (i & 3));
                v = make_uint4(z[0], z[1], z[2], z[3]);
              }
            }
            w[o][half * 4] = v.x, w[o][half * 4 + 1] = v.y, w[o][half * 4 + 2] = v.z, w[o][half * 4 + 3] = v.w;
          }
#pragma unroll
        for (int half = 0; half < 2; ++half) {
          uint4 v = make_uint4(0, 0, 0, 0);
          if (c < x.nt) v = __ldcg(reinterpret_cast<const uint4*>(xs + ch * 32 + half * 16));
          w[kMats][half * 4] = __vsubus4(v.x, less), w[kMats][half * 4 + 1] = __vsubus4(v.y, less);
          w[kMats][half * 4 + 2] = __vsubus4(v.z, less), w[kMats][half * 4 + 3] = __vsubus4(v.w, less);
        }
        if (!(ok = g_wait_warp(&s_sfempty[sfsl], sfph ^ 1u, &s_abort, a.status, 69))) break;
        const uint32_t dst = sf0 + (uint32_t)sfsl * kSfSlot + at;
#pragma unroll
        for (int o = 0; o <= kMats; ++o)
#pragma unroll
          for (int b = 0; b < 8; ++b)
            asm volatile("st.shared.u32 [%0], %1;" ::"r"(dst + (uint32_t)(o * kSfOp + b * kSfTile)), "r"(w[o][b]) : "memory");
        asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
        mbar_arrive(&s_sffull[sfsl]);
        if (++sfsl == kSfRing) sfsl = 0, sfph ^= 1u;
      }
    }
  }
  g_before();
  __syncthreads();
  if (warp == 1) {
    g_after();
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(512u) : "memory");
  }
}

}  // namespace

cudaError_t launch_moe_fp4_factors(const MoeArgs& a, cudaStream_t s) {
  FArgs f;
  f.m = a;
  f.xs = a.xs;
  f.xs_pitch = moe_xs_pitch(a.d_model);
  f.tokens = a.T < kFTokens ? a.T : kFTokens;
  f.stage_bytes = kMats * kFABytes + f.tokens * 1024;
  const int sf = kSfRing * (kMats + 1) * kSfOp;
  f.stages = (kFSmemCap - 1024 - sf) / f.stage_bytes;
  if (f.stages > kFMaxStages) f.stages = kFMaxStages;
  // two accumulators where tensor memory (512 columns) has them beside the scales
  f.acc = f.tokens * 8 < 32 ? 32 : (f.tokens * 8 + 31) / 32 * 32;
  f.nacc = 2 * kMats * f.acc + f.stages * (kMats + 1) * 8 <= 512 ? 2 : 1;
  CUtensorMap m1, m2, mx;
  const uint64_t pitch = (uint64_t)(a.d_model / 2), rows = (uint64_t)a.E * a.d_ff;
  if (!g_map(&m1, a.w1, pitch, rows, kFM) || !g_map(&m2, a.w2, pitch, rows, kFM) ||
      !g_map(&mx, a.xt, pitch, (uint64_t)a.T * 8, 8))
    return cudaErrorInvalidValue;
  const int smem = f.stages * f.stage_bytes + sf + 1024;
  static unsigned configured = 0;
  cudaError_t e = ensure_smem_attr(moe_fp4_factors_kernel, kFSmemCap, &configured);
  if (e != cudaSuccess) return e;
  e = launch_pdl(moe_fp4_factors_kernel, dim3((unsigned)kNumSMs), dim3(kFThreads), (size_t)smem, s, m1, m2, mx, f);
  if (e != cudaSuccess) return e;
  return cudaGetLastError();
}

}  // namespace qs
