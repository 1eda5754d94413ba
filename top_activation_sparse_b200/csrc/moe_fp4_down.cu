// Down projection of 4-bit experts for many tokens, on the tensor cores.
//
//   part[t, c] = sum_{j in a range} h[t, j] s[j, c / 32] q[j, c]
//
// The weights lie neuron by neuron with blocks along the columns: the sum runs
// across their scales, so the block-scaled MMA does not fit.  They are expanded to
// bf16 (exactly) on their way through shared memory and multiplied with h, which
// is the sum of three bf16 numbers, i.e. has its 24 bits (kind::f16, M = 128:
// three rows per token; N = 512 columns, whose sums fill tensor memory).
//   * warp 0 copies the codes of 64 neurons x 512 columns per step, warp 2 the
//     rows of h (2-D TMA, 128-byte swizzle);
//   * warps 3 to 18 expand: a thread takes two blocks of 32 codes (16 bytes each), 20
//     instructions per 8 weights, and stores bf16 rows as the MMA reads them (N
//     contiguous, swizzled).  The columns of a group of 8 are stored in the order
//     0 4 1 5 2 6 3 7: a word's nibbles i and i + 4 make a pair without moves;
//   * one lane of warp 1 issues the MMAs;
//   * the expanding warps add a token's three rows, and what they add up to onto the
//     sums before.
// The tensor core cuts its sums off instead of rounding them, which adds up with their
// number: after sum_steps steps a sum leaves tensor memory, whatever the range's length
// (64 tokens, 16 of 16 experts of 28672 x 1024 each, f32 results: y off by 4.7e-7 of itself with 16
// steps, 8.7e-7 with 32, 7.6e-6 with a whole range of 14336 neurons).
// 32 tokens, 2 of 8 experts of 11008 x 4096 each: 114 us, 1.7 TB/s of the 190 MB (3 us of it per sum).
// Bound by the step's chain: the expansion (1200 cycles of issue) and the MMAs (900)
// overlap, but each hand-over through a barrier takes 300 to 400 cycles while the
// expansion's stores fill the queue that barriers go through.  Smaller steps with four
// places (128 us) and scales through shared memory (114 us) hand over more often.
// (Expanding in registers for mma.sync, 8 tokens at a time: 297 us.)  Every wait is
// bounded.
#include "fp4_mma.cuh"
#include "moe_tables.cuh"

namespace qs {
namespace {

constexpr int kDExpand = 16;                    // warps that expand
constexpr int kDThreads = (3 + kDExpand) * 32;
constexpr int kDK = 64;                         // neurons per step
constexpr int kDCols = kMoeDownCols;            // columns per item
constexpr int kDCodes = kDK * kDCols / 2;       // 16 KB: two boxes of 128 bytes x 64 rows
constexpr int kDB = kDK * kDCols * 2;           // 64 KB: eight boxes of 64 columns x 64 rows
constexpr int kDBox = kDK * 128;                // 8 KB
constexpr int kDA = 128 * kDK * 2;              // 16 KB
constexpr int kDCodeStages = 3;
constexpr int kDAhead = 4;                      // steps by which scales are loaded ahead
constexpr int kDTenth = 10;                     // tokens per 32 rows (30 of them used)
static_assert(kMoeDownTokens == 4 * kDTenth, "four quarters of 10 tokens");
constexpr int kDSmem = 2 * (kDB + kDA) + kDCodeStages * kDCodes + 1024;

// Nibbles c and c + 4 of a word as a pair of bf16.  A code's two exponent bits (bias 1) and
// its mantissa bit, moved to the two lowest exponent bits and the highest mantissa bit of a bf16
// number (bias 127), read as the code's value times 2^-126, subnormal codes too; one product
// brings in 2^126 and the scale.
template <int C, bool BIG>
__device__ __forceinline__ uint32_t d_pair(uint32_t p, uint32_t lo, uint32_t hi) {
  const uint32_t m = C == 0 ? p << 6 : C == 1 ? p << 2 : C == 2 ? p >> 2 : p >> 6;
  const uint32_t s = C == 3 ? p : p << (12 - 4 * C);
  uint32_t v = (m & 0x01c001c0u) | (s & 0x80008000u);
  asm("mul.rn.bf16x2 %0, %0, %1;" : "+r"(v) : "r"(lo));
  if constexpr (BIG) asm("mul.rn.bf16x2 %0, %0, %1;" : "+r"(v) : "r"(hi));
  return v;
}

// a block of 32 codes with scale byte s, to 64 bytes of a row
template <bool BIG>
__device__ __forceinline__ void d_expand(const uint32_t (&v)[4], uint32_t s, uint32_t to, uint32_t part, uint32_t x7) {
  const uint32_t lo = ((!BIG || s < 128u ? s + 126u : 254u) << 7) * 0x10001u;
  const uint32_t hi = (s == 255u ? 0x7fc0u : (s > 128u ? s - 1u : 127u) << 7) * 0x10001u;
#pragma unroll
  for (int c = 0; c < 4; ++c)
    asm volatile("st.shared.v4.u32 [%0], {%1,%2,%3,%4};" ::"r"(to + ((part + (uint32_t)(c << 4)) ^ x7)),
                 "r"(d_pair<0, BIG>(v[c], lo, hi)), "r"(d_pair<1, BIG>(v[c], lo, hi)), "r"(d_pair<2, BIG>(v[c], lo, hi)),
                 "r"(d_pair<3, BIG>(v[c], lo, hi))
                 : "memory");
}

// (an address is added to by one thread only, so that the order is fixed; a reduction at
// L2, for which nothing waits: loading, adding and storing took 30 us per sum more.  Subnormal
// sums count as 0 there)
__device__ __forceinline__ void d_add4(float* p, float x, float y, float z, float w) {
  asm volatile("red.relaxed.gpu.global.add.v4.f32 [%0], {%1, %2, %3, %4};" ::"l"(p), "f"(x), "f"(y), "f"(z), "f"(w) : "memory");
}

__global__ void __launch_bounds__(kDThreads, 1)
    moe_fp4_down_kernel(const __grid_constant__ CUtensorMap map_w, const __grid_constant__ CUtensorMap map_h,
                        const __grid_constant__ MoeArgs a) {
  extern __shared__ __align__(1024) unsigned char smem_raw[];
  __shared__ __align__(8) uint64_t s_cfull[kDCodeStages], s_cempty[kDCodeStages];
  __shared__ __align__(8) uint64_t s_afull[2], s_bfull[2], s_empty[2];
  __shared__ __align__(8) uint64_t s_tfull, s_tempty, s_done;
  __shared__ uint32_t s_tmem;
  __shared__ int s_abort;
  __shared__ MoeTables tb;

  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const uint32_t base = (smem_u32(smem_raw) + 1023u) & ~1023u;
  const uint32_t sa = base + 2 * kDB, scodes = sa + 2 * kDA;
  if (tid == 0) {
    for (int i = 0; i < kDCodeStages; ++i) mbar_init(&s_cfull[i], 1), mbar_init(&s_cempty[i], kDExpand);
    for (int i = 0; i < 2; ++i) mbar_init(&s_afull[i], 1), mbar_init(&s_bfull[i], kDExpand), mbar_init(&s_empty[i], 1);
    mbar_init(&s_tfull, 1);
    mbar_init(&s_tempty, kDExpand);
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
  load_tables(a, tb, kMoeDownTokens, kDThreads);
  g_before();
  __syncthreads();
  g_after();
  const uint32_t tmem = s_tmem;
  const int S = moe_splits(a, tb), items = moe_split_sum(a, tb, S) * a.plan.col_tiles;

  if (warp == 0 || warp == 2) {
    if (lane == 0) {
      // ---- copies: codes (warp 0), h (warp 2) ----
      const bool codes = warp == 0;
      const int stages = codes ? kDCodeStages : 2;
      uint64_t* full = codes ? s_cfull : s_afull;
      uint64_t* empty = codes ? s_cempty : s_empty;
      int n = 0, sl = 0;
      uint32_t ph = 0;
      bool ok = true;
      for (int it = blockIdx.x; it < items && ok; it += gridDim.x) {
        const MoeDownItem d = moe_down_item(a, tb, it, S, kDCols, kDK);
        for (int t0 = 0; t0 < d.cnt && ok; t0 += kMoeDownTokens) {
          const int nt = min(kMoeDownTokens, d.cnt - t0), quarters = (nt + kDTenth - 1) / kDTenth;
          for (int ks = 0; ks < d.steps; ++ks, ++n) {
            if (!(ok = g_wait(&empty[sl], ph ^ 1u, &s_abort, a.status, 90))) break;
            const int j = d.j0 + ks * kDK;
            if (codes) {
              const int boxes = (d.cw + 255) / 256;
              mbar_arrive_expect_tx(&full[sl], (uint32_t)(boxes * kDK * 128));
              for (int b = 0; b < boxes; ++b)
                g_tma(scodes + (uint32_t)(sl * kDCodes + b * kDK * 128), &map_w, d.c0 / 2 + b * 128, d.e * a.d_ff + j, &full[sl]);
            } else {
              mbar_arrive_expect_tx(&full[sl], (uint32_t)(quarters * 32 * 128));
              for (int q = 0; q < quarters; ++q)
                g_tma(sa + (uint32_t)(sl * kDA + q * 32 * 128), &map_h, j, (d.slot0 + t0 + q * kDTenth) * 3, &full[sl]);
            }
            if (++sl == stages) sl = 0, ph ^= 1u;
          }
        }
      }
      // after a give-up: let the copies in flight land
      if (*(volatile int*)&s_abort)
        for (int j = 0; j < stages && j < n; ++j) {
          const int g = n - 1 - j;
          mbar_wait(&full[g % stages], (uint32_t)(g / stages) & 1u);
        }
    }
  } else if (warp == 1) {
    // ---- MMAs.  (The whole warp goes through the steps, one lane issues: what the
    // instructions take is then uniform and need not be moved there lane by lane) ----
    const bool issues = g_elect();
    const uint64_t a0 = g_desc_bf16(sa, 16, 1024), b0 = g_desc_bf16(base, kDBox, 1024);
    int b = 0, piece = 0;
    uint32_t ph = 0;
    bool ok = true;
    for (int it = blockIdx.x; it < items && ok; it += gridDim.x) {
      const MoeDownItem d = moe_down_item(a, tb, it, S, kDCols, kDK);
      for (int t0 = 0; t0 < d.cnt && ok; t0 += kMoeDownTokens) {
        const uint32_t id0 = g_idesc_bf16((uint32_t)min(256, d.cw), 1u), id1 = g_idesc_bf16((uint32_t)max(16, d.cw - 256), 1u);
        for (int ks = 0, in = 0; ks < d.steps; ++ks) {         // in: this step's place in its sum
          if (in == 0 && piece > 0 && !(ok = g_wait_warp(&s_tempty, (uint32_t)(piece - 1) & 1u, &s_abort, a.status, 91))) break;
          // (h has arrived too: the first expanding warp has waited for it)
          if (!(ok = g_wait_warp(&s_bfull[b], ph, &s_abort, a.status, 93))) break;
          g_after();
          const uint64_t ad = a0 + (uint64_t)(b * (kDA / 16)), bd = b0 + (uint64_t)(b * (kDB / 16));
          const bool last = in == a.plan.sum_steps - 1 || ks == d.steps - 1;
          if (issues) {
#pragma unroll
            for (int half = 0; half < 2; ++half) {
              if (half * 256 >= d.cw) break;
#pragma unroll
              for (int kk = 0; kk < kDK / 16; ++kk)
                g_mma_bf16(tmem + half * 256, ad + kk * 2, bd + half * (4 * kDBox / 16) + kk * 128, half ? id1 : id0, in > 0 || kk > 0);
            }
            g_commit(&s_empty[b]);
            if (last) g_commit(&s_tfull);
          }
          __syncwarp();
          if (last) ++piece, in = 0;
          else ++in;
          if ((b ^= 1) == 0) ph ^= 1u;
        }
      }
    }
    if (issues) {
      g_commit(&s_done);                    // every MMA issued has completed when this arrives
      mbar_wait(&s_done, 0u);
    }
    __syncwarp();
  } else {
    // ---- expansion: rows (w & 7) * 8 + lane % 8 of a step, blocks of 32 columns
    // (w >> 3) * 8 + lane / 8 and 4 further ----
    const int w = warp - 3, r = (w & 7) * 8 + (lane & 7), cb = (w >> 3) * 8 + (lane >> 3);
    const int sb = a.d_model / 32;
    const uint32_t x7 = (uint32_t)(r & 7) << 4;
    // codes: 16-byte chunk of the row in its box; bf16: 64 bytes of the row in theirs
    uint32_t src[2], dst[2];
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const int c = cb + 4 * i;
      src[i] = (uint32_t)((c >> 3) * kDK * 128 + r * 128) + ((uint32_t)((c & 7) << 4) ^ x7);
      dst[i] = (uint32_t)((c >> 1) * kDBox + r * 128);
    }
    const uint32_t part = (uint32_t)(cb & 1) << 6;            // which half of the 128 bytes (4 i keeps it)
    int csl = 0, b = 0, piece = 0;
    uint32_t cph = 0, ph = 0;
    bool ok = true;
    for (int it = blockIdx.x; it < items && ok; it += gridDim.x) {
      const MoeDownItem d = moe_down_item(a, tb, it, S, kDCols, kDK);
      const uint8_t* sc = a.sd + ((size_t)d.e * a.d_ff + d.j0 + r) * sb + d.c0 / 32;
      const int left = d.j1 - d.j0 - r;                       // rows from this thread's on
      // scales, some steps ahead of their use (from DRAM)
      uint32_t next[kDAhead][2];
      auto ahead = [&](int ks, uint32_t (&to)[2]) {
#pragma unroll
        for (int i = 0; i < 2; ++i)
          to[i] = ks * kDK < left && (cb + 4 * i) * 32 < d.cw ? (uint32_t)__ldg(sc + (size_t)ks * kDK * sb + cb + 4 * i) : 0u;
      };
      for (int t0 = 0; t0 < d.cnt && ok; t0 += kMoeDownTokens) {
        // results: 10 tokens per quarter of the lanes, three rows each; which lanes the two
        // other rows of this lane's token are in
        const int q = warp & 3, tok = t0 + q * kDTenth + lane / 3;
        const bool mine = lane < 30 && tok < d.cnt;
        const int r3 = lane % 3, from1 = r3 == 0 ? lane + 2 : lane - 1, from2 = r3 == 2 ? lane - 2 : lane + 1;
        float* o = a.parts + ((size_t)d.s * a.T * a.top_k + d.slot0 + (mine ? tok : 0)) * a.d_model + d.c0;
#pragma unroll
        for (int i = 0; i < kDAhead; ++i) ahead(i, next[i]);
        for (int ks = 0, in = 0; ks < d.steps; ++ks) {
          const uint32_t s[2] = {next[0][0], next[0][1]};
          const bool there = ks * kDK < left;
#pragma unroll
          for (int i = 0; i + 1 < kDAhead; ++i) next[i][0] = next[i + 1][0], next[i][1] = next[i + 1][1];
          ahead(ks + kDAhead, next[kDAhead - 1]);
          if (!(ok = g_wait_warp(&s_cfull[csl], cph, &s_empty[b], ph ^ 1u, &s_abort, a.status, 94))) break;
          uint32_t v[2][4];
#pragma unroll
          for (int i = 0; i < 2; ++i)
            asm volatile("ld.shared.v4.u32 {%0,%1,%2,%3}, [%4];"
                         : "=r"(v[i][0]), "=r"(v[i][1]), "=r"(v[i][2]), "=r"(v[i][3])
                         : "r"(scodes + (uint32_t)(csl * kDCodes) + src[i])
                         : "memory");
          // (rows behind the range are 0: what lies there may be anything)
          if (!there) v[0][0] = v[0][1] = v[0][2] = v[0][3] = v[1][0] = v[1][1] = v[1][2] = v[1][3] = 0u;
          // scales above 2 take a second factor (seldom: a warp at a time)
          if (__any_sync(0xffffffffu, max(s[0], s[1]) > 128u)) {
#pragma unroll
            for (int i = 0; i < 2; ++i)
              d_expand<true>(v[i], s[i], base + (uint32_t)(b * kDB) + dst[i], part, x7);
          } else {
#pragma unroll
            for (int i = 0; i < 2; ++i)
              d_expand<false>(v[i], s[i], base + (uint32_t)(b * kDB) + dst[i], part, x7);
          }
          asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
          __syncwarp();
          if (lane == 0) mbar_arrive(&s_cempty[csl]);
          // (one wait per step for the warp that issues the MMAs)
          if (w == 0 && !(ok = g_wait_warp(&s_afull[b], ph, &s_abort, a.status, 92))) break;
          if (lane == 0) mbar_arrive(&s_bfull[b]);
          if (++csl == kDCodeStages) csl = 0, cph ^= 1u;
          if ((b ^= 1) == 0) ph ^= 1u;
          if (++in < a.plan.sum_steps && ks < d.steps - 1) continue;
          in = 0;
          // ---- the sum's results, onto those of the range's sums before it: four
          // warps per quarter of the lanes, 24 columns in turn, of which each of a token's three
          // lanes adds up 8 (two shuffles for three columns: a quarter's warps share one
          // scheduler, whose shuffles take four cycles each) ----
          if (!(ok = g_wait_warp(&s_tfull, (uint32_t)piece++ & 1u, &s_abort, a.status, 96))) break;
          g_after();
          if (t0 + q * kDTenth < d.cnt)
            for (int c = (w >> 2) * 24; c < d.cw; c += kDExpand / 4 * 24) {
              uint32_t u[3][8];
#pragma unroll
              for (int g = 0; g < 3; ++g)
                if (c + 8 * g < kDCols) g_ld8(tmem + ((uint32_t)(q * 32) << 16) + (uint32_t)(c + 8 * g), u[g]);
              g_ld_wait();
              float y[8];
#pragma unroll
              for (int i = 0; i < 8; ++i) {
                const uint32_t own = r3 == 0 ? u[0][i] : r3 == 1 ? u[1][i] : u[2][i];
                const uint32_t one = r3 == 0 ? u[1][i] : r3 == 1 ? u[2][i] : u[0][i];
                const uint32_t two = r3 == 0 ? u[2][i] : r3 == 1 ? u[0][i] : u[1][i];
                y[i] = (__uint_as_float(__shfl_sync(0xffffffffu, one, from1)) + __uint_as_float(__shfl_sync(0xffffffffu, two, from2))) +
                       __uint_as_float(own);
              }
              if (mine && c + 8 * r3 < d.cw) {
                float* to = o + c + 8 * r3;
                if (ks >= a.plan.sum_steps) {
                  d_add4(to, y[0], y[2], y[4], y[6]);
                  d_add4(to + 4, y[1], y[3], y[5], y[7]);
                } else {
                  __stcg(reinterpret_cast<float4*>(to), make_float4(y[0], y[2], y[4], y[6]));
                  __stcg(reinterpret_cast<float4*>(to) + 1, make_float4(y[1], y[3], y[5], y[7]));
                }
              }
            }
          g_before();
          __syncwarp();
          if (lane == 0) mbar_arrive(&s_tempty);
        }
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

// y from the partial sums, in the order of the ranges and then of the choices:
// 4 outputs per thread.
constexpr int kSThreads = 128;
__global__ void __launch_bounds__(kSThreads) moe_sum_kernel(const __grid_constant__ MoeArgs a) {
  __shared__ MoeTables tb;
  pdl_begin();
  load_tables(a, tb, kMoeDownTokens, kSThreads);
  __syncthreads();
  const int S = moe_splits(a, tb), n4 = a.d_model / 4;
  const long long i = (long long)blockIdx.x * kSThreads + threadIdx.x;
  if (i >= (long long)a.T * n4) return;
  const int t = (int)(i / n4), c = (int)(i - (long long)t * n4) * 4;
  const size_t slots = (size_t)a.T * a.top_k;
  float4 y = make_float4(0, 0, 0, 0);
  for (int j = 0; j < a.top_k; ++j) {
    const int slot = __ldcg(a.table + kMtSlot + t * a.top_k + j);
    const float p = __ldcg(a.share + t * a.top_k + j);
    int ai = 0;
    for (int step = kMoeMaxE / 2; step; step >>= 1)
      if (ai + step < tb.active && tb.first[ai + step] <= slot) ai += step;
    const int n = moe_expert_splits(a, tb, ai, S);
    const float* src = a.parts + (size_t)slot * a.d_model + c;
    float4 v = make_float4(0, 0, 0, 0);
#pragma unroll 4
    for (int s = 0; s < n; ++s) {
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

}  // namespace

cudaError_t launch_moe_sum(const MoeArgs& a, cudaStream_t s) {
  const size_t blocks = ((size_t)a.T * (a.d_model / 4) + kSThreads - 1) / kSThreads;
  const cudaError_t e = launch_pdl(moe_sum_kernel, dim3((unsigned)blocks), dim3(kSThreads), 0, s, a);
  if (e != cudaSuccess) return e;
  return cudaGetLastError();
}

cudaError_t launch_moe_fp4_down(const MoeArgs& a, cudaStream_t s) {
  CUtensorMap mw, mh;
  if (!g_map(&mw, a.wd, (uint64_t)(a.d_model / 2), (uint64_t)a.E * a.d_ff, kDK)) return cudaErrorInvalidValue;
  auto fn = g_encode_fn();
  cuuint64_t dims[2] = {(cuuint64_t)a.d_ff, (cuuint64_t)a.T * a.top_k * 3};
  cuuint64_t strides[1] = {(cuuint64_t)a.d_ff * 2};
  cuuint32_t box[2] = {kDK, 32}, estr[2] = {1, 1};
  if (fn(&mh, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 2, a.h, dims, strides, box, estr, CU_TENSOR_MAP_INTERLEAVE_NONE,
         CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) != CUDA_SUCCESS)
    return cudaErrorInvalidValue;
  static unsigned configured = 0;
  cudaError_t e = ensure_smem_attr(moe_fp4_down_kernel, kDSmem, &configured);
  if (e != cudaSuccess) return e;
  e = launch_pdl(moe_fp4_down_kernel, dim3((unsigned)kNumSMs), dim3(kDThreads), (size_t)kDSmem, s, mw, mh, a);
  if (e != cudaSuccess) return e;
  return cudaGetLastError();
}

}  // namespace qs
