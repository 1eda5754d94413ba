// bf16 experts for several tokens on the tensor cores: h, and the down projection's
// partial sums.
//
//   v[t, j] = sum_i W[e][j, i] x[t, i] (both matrices),  h = act(v_gate, v_up)
//   part[t, c] = sum_{j in a range} h[t, j] W_down[e][j, c]
//
// Bound by the weights' bytes, all of which are read: where several tokens share an
// expert, few neurons are closed for all of them, and one pass of TMA tiles outruns
// the gathered rows and the repeated passes of moe_kernel.cuh (8 experts of 11008 x 4096, 2
// per token, squared ReLU: 8 tokens, 7 experts used, 317 against 418 us; 64 tokens 372 against
// 994, the weights' 2.16 GB at 5.8 TB/s).
//   * factors: 128 neurons of both matrices are the MMA's M side, all tokens of the
//     launch its N side (up to 64: their products cost less than the copies, and
//     the step's x is one tile); a result warp picks its expert's tokens;
//   * down: h, the sum of three bf16 numbers, is the M side (three rows per token, 10
//     tokens per 32 lanes), 256 columns of the weights' rows the N side, read as they
//     lie (N contiguous).  Ranges are whole steps of 64 neurons; the rows behind an
//     expert's last are out of the tensor map's range and read as 0.
// The tensor core cuts its sums off instead of rounding them, which adds up with their
// number: after 128 inputs (or neurons) a sum goes to registers, where the sums are
// added in float32 (one sum over 4096 inputs and 11008 neurons: y off by 1.8e-5 of itself;
// after every 256: 1.2e-6).
// One warp copies (2-D and 3-D TMA, 128-byte swizzle), one lane of another issues the
// MMAs, the others read the sums.  Every wait is bounded.
#include "fp4_mma.cuh"
#include "moe_tables.cuh"

namespace qs {
namespace {

constexpr int kTThreads = 192, kTDThreads = 320; // factors; down
constexpr int kTChunk = 2;                      // steps per sum
constexpr int kTK = 64;                         // inputs, or neurons, per step: 128-byte rows
constexpr int kTM = 128;                        // neurons per unit
constexpr int kTW = kTM * kTK * 2;              // 16 KB
constexpr int kTMaxStages = 8;
constexpr int kTSmemCap = 216 * 1024;
constexpr int kTCols = kMoeDownColsBf16;        // columns of the down projection per item
constexpr int kTB = kTK * kTCols * 2;           // 32 KB: four boxes of 64 columns x 64 rows
constexpr int kTBox = kTK * 128;
constexpr int kTA = 128 * kTK * 2;              // 16 KB: h
constexpr int kTTenth = 10;                     // tokens per 32 rows of h
static_assert(kMoeDownTokens == 4 * kTTenth, "four quarters of 10 tokens");

__device__ __forceinline__ void t_tma3(uint32_t dst, const CUtensorMap* map, int x, int y, int z, uint64_t* bar) {
  asm volatile(
      "cp.async.bulk.tensor.3d.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
      " [%0], [%1, {%2, %3, %4}], [%5];" ::"r"(dst),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(x), "r"(y), "r"(z), "r"(smem_u32(bar))
      : "memory");
}
// 16 columns more onto s
__device__ __forceinline__ void t_add16(uint32_t taddr, float* s) {
  uint32_t u[2][8];
  g_ld8(taddr, u[0]);
  g_ld8(taddr + 8, u[1]);
  g_ld_wait();
#pragma unroll
  for (int i = 0; i < 16; ++i) s[i] += __uint_as_float(u[i >> 3][i & 7]);
}

struct TShared {
  uint64_t full[kTMaxStages], empty[kTMaxStages], tfull[2], tempty[2], done;
  int16_t place[4][kMoeMaxT];                   // a result warp's: a token's place among its expert's, or -1
  uint32_t tmem;
  int abort;
  MoeTables tb;
};

__device__ __forceinline__ void t_begin(TShared& s, int stages, int readers) {
  if (threadIdx.x == 0) {
    for (int i = 0; i < stages; ++i) mbar_init(&s.full[i], 1), mbar_init(&s.empty[i], 1);
    for (int i = 0; i < 2; ++i) mbar_init(&s.tfull[i], 1), mbar_init(&s.tempty[i], readers);
    mbar_init(&s.done, 1);
    mbar_fence_init();
    s.abort = 0;
  }
  if (threadIdx.x >> 5 == 1) {
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_u32(&s.tmem)), "r"(512u)
                 : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
  }
}
__device__ __forceinline__ void t_end(TShared& s) {
  g_before();
  __syncthreads();
  if (threadIdx.x >> 5 == 1) {
    g_after();
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(s.tmem), "r"(512u) : "memory");
  }
}
// after a give-up: let the copies in flight land (n were sent)
__device__ __forceinline__ void t_land(TShared& s, int stages, int n) {
  if (*(volatile int*)&s.abort)
    for (int j = 0; j < stages && j < n; ++j) {
      const int g = n - 1 - j;
      mbar_wait(&s.full[g % stages], (uint32_t)(g / stages) & 1u);
    }
}

struct TArgs {
  MoeArgs m;
  int rows;                                     // tokens in x's tile (a multiple of 16)
  int stages, stage_bytes;
};

// ROWS: f.rows, or more
template <int ROWS>
__global__ void __launch_bounds__(kTThreads, 1)
    moe_bf16_factors_kernel(const __grid_constant__ CUtensorMap map_1, const __grid_constant__ CUtensorMap map_2,
                            const __grid_constant__ CUtensorMap map_x, const __grid_constant__ TArgs f) {
  extern __shared__ __align__(1024) unsigned char smem_raw[];
  __shared__ __align__(8) TShared s;
  const MoeArgs& a = f.m;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const uint32_t base = (smem_u32(smem_raw) + 1023u) & ~1023u;
  const int nk = (a.d_model + kTK - 1) / kTK, mtiles = (a.d_ff + kTM - 1) / kTM;
  t_begin(s, f.stages, 4);
  pdl_begin();
  load_tables(a, s.tb, kMoeMaxT, kTThreads);
  g_before();
  __syncthreads();
  g_after();
  const uint32_t tmem = s.tmem;
  const int units = s.tb.active * mtiles;
  if (warp == 0) {
    if (lane == 0) {
      int n = 0, sl = 0;
      uint32_t ph = 0;
      bool ok = true;
      for (int u = blockIdx.x; u < units && ok; u += gridDim.x) {
        const int row = s.tb.expert[u / mtiles] * a.d_ff + u % mtiles * kTM;
        for (int ks = 0; ks < nk; ++ks, ++n) {
          if (!(ok = g_wait(&s.empty[sl], ph ^ 1u, &s.abort, a.status, 100))) break;
          const uint32_t st = base + (uint32_t)(sl * f.stage_bytes);
          mbar_arrive_expect_tx(&s.full[sl], (uint32_t)(2 * kTW + f.rows * 128));
          g_tma(st, &map_1, ks * kTK, row, &s.full[sl]);
          g_tma(st + kTW, &map_2, ks * kTK, row, &s.full[sl]);
          g_tma(st + 2 * kTW, &map_x, ks * kTK, 0, &s.full[sl]);
          if (++sl == f.stages) sl = 0, ph ^= 1u;
        }
      }
      t_land(s, f.stages, n);
    }
  } else if (warp == 1) {
    const bool issues = g_elect();
    const uint32_t id = g_idesc_bf16((uint32_t)f.rows, 0u);
    const uint64_t d0 = g_desc_bf16(base, 16, 1024);
    int sl = 0, piece = 0;
    uint32_t ph = 0;
    bool ok = true;
    for (int u = blockIdx.x; u < units && ok; u += gridDim.x) {
      for (int ks = 0; ks < nk; ++ks) {
        const int ab = piece & 1;
        if (ks % kTChunk == 0 && piece >= 2 && !(ok = g_wait_warp(&s.tempty[ab], (uint32_t)(piece / 2 - 1) & 1u, &s.abort, a.status, 101)))
          break;
        if (!(ok = g_wait_warp(&s.full[sl], ph, &s.abort, a.status, 102))) break;
        g_after();
        const uint64_t st = d0 + (uint64_t)(sl * (f.stage_bytes / 16));
        const bool last = ks % kTChunk == kTChunk - 1 || ks == nk - 1;
        if (issues) {
#pragma unroll
          for (int kk = 0; kk < kTK / 16; ++kk)
#pragma unroll
            for (int o = 0; o < 2; ++o)
              g_mma_bf16(tmem + ab * 128 + o * 64, st + o * (kTW / 16) + kk * 2, st + 2 * (kTW / 16) + kk * 2, id,
                    ks % kTChunk > 0 || kk > 0);
          g_commit(&s.empty[sl]);
          if (last) g_commit(&s.tfull[ab]);
        }
        __syncwarp();
        if (last) ++piece;
        if (++sl == f.stages) sl = 0, ph ^= 1u;
      }
    }
    if (issues) {
      g_commit(&s.done);                    // every MMA issued has completed when this arrives
      mbar_wait(&s.done, 0u);
    }
    __syncwarp();
  } else {
    const int q = warp & 3;
    int16_t* place = s.place[q];
    int piece = 0;
    bool ok = true;
    for (int u = blockIdx.x; u < units && ok; u += gridDim.x) {
      const int ai = u / mtiles, j = u % mtiles * kTM + q * 32 + lane;
      const int e = s.tb.expert[ai], first = s.tb.first[ai], cnt = s.tb.count[ai];
      const bool mine = j < a.d_ff;
      const size_t bi = (size_t)e * a.d_ff + (mine ? j : 0);
      const float b1 = a.b1 ? __ldg(a.b1 + bi) : 0.0f, b2 = a.b2 ? __ldg(a.b2 + bi) : 0.0f;
      place[lane] = place[lane + 32] = -1;
      __syncwarp();
      for (int c = lane; c < cnt; c += 32) place[s.tb.token[first + c]] = (int16_t)c;
      __syncwarp();
      float v[2][ROWS];
#pragma unroll
      for (int t = 0; t < ROWS; ++t) v[0][t] = v[1][t] = 0.0f;
      for (int ks = 0; ks < nk; ks += kTChunk, ++piece) {
        const int ab = piece & 1;
        if (!(ok = g_wait_warp(&s.tfull[ab], (uint32_t)(piece / 2) & 1u, &s.abort, a.status, 103))) break;
        g_after();
        const uint32_t acc = tmem + ((uint32_t)(q * 32) << 16) + (uint32_t)(ab * 128);
#pragma unroll
        for (int t = 0; t < ROWS; t += 16)
          if (t < f.rows) {
            t_add16(acc + t, &v[0][t]);
            t_add16(acc + 64 + t, &v[1][t]);
          }
        g_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(&s.tempty[ab]);
      }
      if (!ok) break;
#pragma unroll
      for (int t = 0; t < ROWS; ++t) {
        const int c = place[t];
        if (c < 0) continue;
        float h = relu_nan(v[0][t] + b1), g = v[1][t] + b2;
        if (!a.drelu) h *= h;
        else g = relu_nan(g);
        // (a closed first factor is 0 whatever the other is)
        h = h == 0.0f ? 0.0f : h * g;
        // h as the sum of three bf16 numbers (an infinity or a NaN has no rest)
        __nv_bfloat16* o = reinterpret_cast<__nv_bfloat16*>(a.h) + (size_t)(first + c) * 3 * a.d_ff + j;
        const bool finite = fabsf(h) <= 3.0e38f;
#pragma unroll
        for (int i = 0; i < 3; ++i) {
          const __nv_bfloat16 b = __float2bfloat16_rn(h);
          if (mine) o[(size_t)i * a.d_ff] = b;
          h = finite ? h - __bfloat162float(b) : 0.0f;
        }
      }
      __syncwarp();
    }
  }
  t_end(s);
}

__global__ void __launch_bounds__(kTDThreads, 1)
    moe_bf16_down_kernel(const __grid_constant__ CUtensorMap map_w, const __grid_constant__ CUtensorMap map_h,
                         const __grid_constant__ TArgs f) {
  extern __shared__ __align__(1024) unsigned char smem_raw[];
  __shared__ __align__(8) TShared s;
  const MoeArgs& a = f.m;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const uint32_t base = (smem_u32(smem_raw) + 1023u) & ~1023u;
  t_begin(s, f.stages, 8);
  pdl_begin();
  load_tables(a, s.tb, kMoeDownTokens, kTDThreads);
  g_before();
  __syncthreads();
  g_after();
  const uint32_t tmem = s.tmem;
  const int S = moe_splits(a, s.tb), items = moe_split_sum(a, s.tb, S) * a.plan.col_tiles;
  if (warp == 0) {
    if (lane == 0) {
      int n = 0, sl = 0;
      uint32_t ph = 0;
      bool ok = true;
      for (int it = blockIdx.x; it < items && ok; it += gridDim.x) {
        const MoeDownItem d = moe_down_item(a, s.tb, it, S, kTCols, kTK);
        const int boxes = (d.cw + 63) / 64;
        for (int t0 = 0; t0 < d.cnt && ok; t0 += kMoeDownTokens) {
          const int quarters = (min(kMoeDownTokens, d.cnt - t0) + kTTenth - 1) / kTTenth;
          for (int ks = 0; ks < d.steps; ++ks, ++n) {
            if (!(ok = g_wait(&s.empty[sl], ph ^ 1u, &s.abort, a.status, 104))) break;
            const int j = d.j0 + ks * kTK;
            const uint32_t st = base + (uint32_t)(sl * f.stage_bytes);
            mbar_arrive_expect_tx(&s.full[sl], (uint32_t)(boxes * kTBox + quarters * 32 * 128));
            for (int b = 0; b < boxes; ++b) t_tma3(st + b * kTBox, &map_w, d.c0 + b * 64, j, d.e, &s.full[sl]);
            for (int q = 0; q < quarters; ++q)
              g_tma(st + kTB + q * 32 * 128, &map_h, j, (d.slot0 + t0 + q * kTTenth) * 3, &s.full[sl]);
            if (++sl == f.stages) sl = 0, ph ^= 1u;
          }
        }
      }
      t_land(s, f.stages, n);
    }
  } else if (warp == 1) {
    const bool issues = g_elect();
    const uint64_t a0 = g_desc_bf16(base + kTB, 16, 1024), b0 = g_desc_bf16(base, kTBox, 1024);
    int sl = 0, piece = 0;
    uint32_t ph = 0;
    bool ok = true;
    for (int it = blockIdx.x; it < items && ok; it += gridDim.x) {
      const MoeDownItem d = moe_down_item(a, s.tb, it, S, kTCols, kTK);
      const uint32_t id = g_idesc_bf16((uint32_t)d.cw, 1u);
      for (int t0 = 0; t0 < d.cnt && ok; t0 += kMoeDownTokens)
        for (int ks = 0; ks < d.steps; ++ks) {
          const int ab = piece & 1;
          if (ks % kTChunk == 0 && piece >= 2 &&
              !(ok = g_wait_warp(&s.tempty[ab], (uint32_t)(piece / 2 - 1) & 1u, &s.abort, a.status, 105)))
            break;
          if (!(ok = g_wait_warp(&s.full[sl], ph, &s.abort, a.status, 106))) break;
          g_after();
          const uint64_t ad = a0 + (uint64_t)(sl * (f.stage_bytes / 16)), bd = b0 + (uint64_t)(sl * (f.stage_bytes / 16));
          const bool last = ks % kTChunk == kTChunk - 1 || ks == d.steps - 1;
          if (issues) {
#pragma unroll
            for (int kk = 0; kk < kTK / 16; ++kk)
              g_mma_bf16(tmem + ab * 256, ad + kk * 2, bd + kk * 128, id, ks % kTChunk > 0 || kk > 0);
            g_commit(&s.empty[sl]);
            if (last) g_commit(&s.tfull[ab]);
          }
          __syncwarp();
          if (last) ++piece;
          if (++sl == f.stages) sl = 0, ph ^= 1u;
        }
    }
    if (issues) {
      g_commit(&s.done);
      mbar_wait(&s.done, 0u);
    }
    __syncwarp();
  } else {
    // two warps per 32 lanes, 128 columns each
    const int q = warp & 3, half = (warp - 2) >> 2 << 7;
    const size_t slots = (size_t)a.T * a.top_k;
    int piece = 0;
    bool ok = true;
    for (int it = blockIdx.x; it < items && ok; it += gridDim.x) {
      const MoeDownItem d = moe_down_item(a, s.tb, it, S, kTCols, kTK);
      for (int t0 = 0; t0 < d.cnt && ok; t0 += kMoeDownTokens) {
        const int tok = t0 + q * kTTenth + lane / 3;
        const bool used = t0 + q * kTTenth < d.cnt, mine = lane < 30 && lane % 3 == 0 && tok < d.cnt;
        float y[128];
#pragma unroll
        for (int i = 0; i < 128; ++i) y[i] = 0.0f;
        for (int ks = 0; ks < d.steps; ks += kTChunk, ++piece) {
          const int ab = piece & 1;
          if (!(ok = g_wait_warp(&s.tfull[ab], (uint32_t)(piece / 2) & 1u, &s.abort, a.status, 107))) break;
          g_after();
          if (used) {
            const uint32_t acc = tmem + ((uint32_t)(q * 32) << 16) + (uint32_t)(ab * 256 + half);
#pragma unroll
            for (int c = 0; c < 128; c += 16)
              if (half + c < d.cw) t_add16(acc + (uint32_t)c, y + c);
          }
          g_before();
          __syncwarp();
          if (lane == 0) mbar_arrive(&s.tempty[ab]);
        }
        if (!ok || !used) continue;
        float* o = a.parts + ((size_t)d.s * slots + d.slot0 + (mine ? tok : 0)) * a.d_model + d.c0 + half;
#pragma unroll
        for (int c = 0; c < 128; c += 4) {
          if (half + c >= d.cw) break;
          float4 z;
          float* zz = reinterpret_cast<float*>(&z);
#pragma unroll
          for (int i = 0; i < 4; ++i)
            zz[i] = (__shfl_down_sync(0xffffffffu, y[c + i], 2) + __shfl_down_sync(0xffffffffu, y[c + i], 1)) + y[c + i];
          if (mine) __stcg(reinterpret_cast<float4*>(o + c), z);
        }
      }
    }
  }
  t_end(s);
}

// bf16 [z][rows][cols]: box of 64 columns x box_rows (x 1)
bool t_map(CUtensorMap* m, const void* ptr, uint64_t cols, uint64_t rows, uint64_t z, uint32_t box_rows) {
  auto fn = g_encode_fn();
  if (fn == nullptr) return false;
  cuuint64_t dims[3] = {cols, rows, z};
  cuuint64_t strides[2] = {cols * 2, cols * rows * 2};
  cuuint32_t box[3] = {kTK, box_rows, 1}, estr[3] = {1, 1, 1};
  return fn(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, z ? 3 : 2, const_cast<void*>(ptr), dims, strides, box, estr,
            CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
            CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

}  // namespace

cudaError_t launch_moe_bf16_tensor(const MoeArgs& a, cudaStream_t s) {
  static unsigned done_f[3] = {0, 0, 0}, done_d = 0;
  CUtensorMap m1, m2, mx, mw, mh;
  TArgs f;
  f.m = a;
  f.rows = (a.T + 15) / 16 * 16;
  f.stage_bytes = 2 * kTW + f.rows * 128;
  f.stages = (kTSmemCap - 1024) / f.stage_bytes;
  if (f.stages > kTMaxStages) f.stages = kTMaxStages;
  const uint64_t dm = (uint64_t)a.d_model, dff = (uint64_t)a.d_ff, E = (uint64_t)a.E;
  if (!t_map(&m1, a.w1, dm, E * dff, 0, kTM) || !t_map(&m2, a.w2, dm, E * dff, 0, kTM) ||
      !t_map(&mx, a.x, dm, (uint64_t)a.T, 0, (uint32_t)f.rows) || !t_map(&mw, a.wd, dm, dff, E, kTK) ||
      !t_map(&mh, a.h, dff, (uint64_t)a.T * a.top_k * 3, 0, 32))
    return cudaErrorInvalidValue;
  auto factors = [&](auto kernel, unsigned* done) {
    const cudaError_t r = ensure_smem_attr(kernel, kTSmemCap, done);
    if (r != cudaSuccess) return r;
    return launch_pdl(kernel, dim3((unsigned)kNumSMs), dim3(kTThreads), (size_t)(f.stages * f.stage_bytes + 1024), s, m1, m2, mx, f);
  };
  cudaError_t e = ensure_smem_attr(moe_bf16_down_kernel, kTSmemCap, &done_d);
  if (e != cudaSuccess) return e;
  e = f.rows == 16 ? factors(moe_bf16_factors_kernel<16>, &done_f[0])
                   : f.rows == 32 ? factors(moe_bf16_factors_kernel<32>, &done_f[1]) : factors(moe_bf16_factors_kernel<64>, &done_f[2]);
  if (e != cudaSuccess) return e;
  f.stage_bytes = kTB + kTA;
  f.stages = (kTSmemCap - 1024) / f.stage_bytes;
  e = launch_pdl(moe_bf16_down_kernel, dim3((unsigned)kNumSMs), dim3(kTDThreads), (size_t)(f.stages * f.stage_bytes + 1024), s, mw,
                 mh, f);
  if (e != cudaSuccess) return e;
  return cudaGetLastError();
}

}  // namespace qs
