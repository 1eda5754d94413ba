// Product of two microscaled 4-bit matrices on the 5th-generation tensor cores
// (tcgen05.mma with block scales, accumulators and scales in tensor memory).
//
//   y[t, j] = g_x g_w sum_b sx[t, b] sw[j, b] sum_{i in block b} qx[t, i] qw[j, i]
//
// A product of two e2m1 numbers is a multiple of 1/4 of at most 36, so a
// block's sum is exact; the scaled sums are added in float32.
//
// The weight is the MMA's M side (tiles of 128 outputs), the tokens are its N side
// (8 to 128): a few tokens then cost what the weight's bytes cost.  (Many tokens:
// fp4_gemm_wide.cu.)
//   * warp 0 copies steps of 256 inputs into a ring: 128 weight rows and the
//     tile's tokens (128-byte rows, 128-byte swizzle, 2-D TMA) and the scales'
//     512-byte tiles (plain bulk copies; their layout in global memory is the
//     one tensor memory wants).  The weights of the first steps are asked for
//     before the kernel waits for the one that quantises x: they do not depend
//     on it.
//   * one thread of warp 1 copies a step's scales to tensor memory
//     (tcgen05.cp, one 512-byte tile per 4 columns, a place of its own per ring
//     stage: the commit that frees the stage frees both) and issues its four
//     MMAs of K = 64.
//   * warps 2 to 5 read the accumulator and store y, column by token.
// Where the tiles are fewer than the SMs, a cluster of up to 8 CTAs shares a
// tile's steps: each leaves its partial sums in its own shared memory, and
// after a cluster barrier each adds a slice of them over the cluster, in the
// order of the steps (results do not depend on timing, and no partial sum
// leaves the chip).  An earlier form dealt the steps of all tiles out evenly
// over 148 CTAs with the partial sums in global memory, handed over by
// tickets: its fences, tickets and re-reads cost more than the data (the whole call,
// 8 tokens, NV, 11008 -> 4096 dense: 23.5 us against 15.2 now; the weight alone takes
// 4.0 at the memory's rate.  What is left is latency: quantisation 2 us, launch, the first
// steps' copies, two cluster barriers).  Every wait is bounded.
#include <mutex>

#include "fp4.cuh"
#include "fp4_mma.cuh"

namespace qs {
namespace {

constexpr int kGThreads = 192;
constexpr int kGM = 128;                 // outputs per tile
constexpr int kGABytes = kGM * kGK / 2;  // 16 KB
constexpr int kGSmemCap = 222 * 1024;

constexpr int gmin(int a, int b) { return a < b ? a : b; }

template <bool NV, int NT>
struct GShape {
  static constexpr int kAtoms = kGK / (NV ? 16 : 32) / 4;    // 512-byte scale tiles per step (4 / 2)
  static constexpr int kB = NT * kGK / 2;
  static constexpr int kSfA = kAtoms * kSfTile;
  static constexpr int kSfB = kAtoms * kSfTile;
  static constexpr int kStage = kGABytes + kB + kSfA + kSfB;
  static constexpr int kAcc = NT < 32 ? 32 : NT;             // accumulator columns (allocated)
  static constexpr int kNacc = 2;                            // accumulators
  static constexpr int kSfCols = kAtoms * 8;                 // tensor-memory columns per stage
  static constexpr int kStages = gmin((kGSmemCap - 1024) / kStage, (512 - kNacc * kAcc) / kSfCols);
  static constexpr int kSmem = kStages * kStage + 1024;
  static_assert(kStage % 1024 == 0, "the swizzled tiles start on 1 KB");
  static_assert(kStages >= 3, "ring too short");
};

// instruction descriptor of the block-scaled 4-bit MMA: A and B e2m1, both
// K-major, f32 accumulators, M = 128, N = NT; scale type e8m0 (1) or e4m3 (0);
// MX: which half of the 4 scale bytes (0 or 2) this K = 64 takes
template <bool NV, int NT>
__device__ constexpr uint32_t g_idesc(uint32_t sf_id) {
  return (sf_id << 4) | (1u << 7) | (1u << 10) | ((uint32_t)(NT >> 3) << 17) |
         ((NV ? 0u : 1u) << 23) | ((uint32_t)(kGM >> 4) << 24) | (sf_id << 29);
}

// A CTA's steps in order: with one CTA per tile the whole tiles blockIdx.x +
// i * gridDim.x, else its share of its cluster's tile.
struct GWalk {
  int nk, ntiles, stride;
  int tile, ks, mt, nt;
  __device__ GWalk(const Fp4GemmPlan& P)
      : nk(P.nk), ntiles(P.ntiles), stride((int)gridDim.x) {
    tile = (int)blockIdx.x / P.cluster;
    ks = P.cluster > 1 ? first_step(P, (int)blockIdx.x % P.cluster) : 0;
    place();
  }
  __device__ static int first_step(const Fp4GemmPlan& P, int rank) { return P.nk * rank / P.cluster; }
  __device__ void place() { mt = tile / ntiles, nt = tile - mt * ntiles; }
  __device__ void next() {
    if (++ks == nk) ks = 0, tile += stride, place();
  }
};

__device__ __forceinline__ void g_store(const Fp4GemmArgs& a, size_t o, float f, bool nv, float scale) {
  if (nv) f = __fmul_rn(f, scale);
  if (a.y_bf16) reinterpret_cast<__nv_bfloat16*>(a.y)[o] = __float2bfloat16_rn(f);
  else reinterpret_cast<float*>(a.y)[o] = f;
}

template <bool NV, int NT>
__global__ void __launch_bounds__(kGThreads, 1)
    fp4_gemm_kernel(const __grid_constant__ CUtensorMap map_w, const __grid_constant__ CUtensorMap map_x,
                    Fp4GemmArgs a) {
  using S = GShape<NV, NT>;
  extern __shared__ __align__(1024) unsigned char smem_raw[];
  __shared__ __align__(8) uint64_t s_full[S::kStages];
  __shared__ __align__(8) uint64_t s_empty[S::kStages];
  __shared__ __align__(8) uint64_t s_tfull[2], s_tempty[2];
  __shared__ __align__(8) uint64_t s_done;
  __shared__ uint32_t s_tmem;
  __shared__ int s_abort;

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const uint32_t base = (smem_u32(smem_raw) + 1023u) & ~1023u;
  const Fp4GemmPlan& P = a.plan;
  const int nk = P.nk;
  const int tiles = P.mtiles * P.ntiles;
  const int nblocks = a.d_in / (NV ? 16 : 32);
  const size_t tpr = fp4_tiles_per_row(nblocks);
  const int C = P.cluster, rank = (int)blockIdx.x % C;
  const int n = C > 1 ? GWalk::first_step(P, rank + 1) - GWalk::first_step(P, rank)
                      : ((tiles - 1 - (int)blockIdx.x) / (int)gridDim.x + 1) * nk;   // this CTA's steps

  if (threadIdx.x == 0) {
    for (int i = 0; i < S::kStages; ++i) {
      mbar_init(&s_full[i], 1);
      mbar_init(&s_empty[i], 1);
    }
    for (int b = 0; b < 2; ++b) {
      mbar_init(&s_tfull[b], 1);
      mbar_init(&s_tempty[b], 4);
    }
    mbar_init(&s_done, 1);
    mbar_fence_init();
    s_abort = 0;
  }
  if (warp == 1) {
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_u32(&s_tmem)), "r"(512u)
                 : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
  }
  g_before();
  __syncthreads();
  g_after();
  const uint32_t tmem = s_tmem;
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");

  float scale = 1.0f;                       // the NV form's tensor scales

  if (warp == 0) {
    if (lane == 0) {
      // ---- copies ----
      // a row's last step may have fewer scale tiles
      auto atoms_at = [&](int ks) { return gmin(S::kAtoms, (int)tpr - ks * S::kAtoms); };
      auto copy_w = [&](const GWalk& w, int sl) {
        const int at = atoms_at(w.ks);
        const uint32_t st = base + (uint32_t)(sl * S::kStage);
        mbar_arrive_expect_tx(&s_full[sl], (uint32_t)(kGABytes + S::kB + 2 * at * kSfTile));
        g_tma(st, &map_w, w.ks * (kGK / 2), w.mt * kGM, &s_full[sl]);
        g_bulk(st + kGABytes + S::kB, a.ws + ((size_t)w.mt * tpr + (size_t)w.ks * S::kAtoms) * kSfTile,
               (uint32_t)(at * kSfTile), &s_full[sl]);
      };
      auto copy_x = [&](const GWalk& w, int sl) {
        const int at = atoms_at(w.ks);
        const uint32_t st = base + (uint32_t)(sl * S::kStage);
        g_tma(st + kGABytes, &map_x, w.ks * (kGK / 2), w.nt * NT, &s_full[sl]);
        g_bulk(st + kGABytes + S::kB + S::kSfA, a.xs + ((size_t)w.nt * tpr + (size_t)w.ks * S::kAtoms) * kSfTile,
               (uint32_t)(at * kSfTile), &s_full[sl]);
      };
      const int head = n < S::kStages ? n : S::kStages;
      GWalk w(P), wx(P);
      for (int i = 0; i < head; ++i, w.next()) copy_w(w, i);
      asm volatile("griddepcontrol.wait;" ::: "memory");
      for (int i = 0; i < head; ++i, wx.next()) copy_x(wx, i);
      int i = head;
      for (int sl = 0, ph = 0; i < n; ++i, w.next()) {
        if (!g_wait(&s_empty[sl], (uint32_t)ph, &s_abort, a.status, 60)) break;
        copy_w(w, sl);
        copy_x(w, sl);
        if (++sl == S::kStages) sl = 0, ph ^= 1;
      }
      // after a give-up: let the copies in flight land
      if (*(volatile int*)&s_abort)
        for (int j = 0; j < S::kStages && j < i; ++j) {
          const int g = i - 1 - j;
          mbar_wait(&s_full[g % S::kStages], (uint32_t)(g / S::kStages) & 1u);
        }
    }
  } else if (warp == 1) {
    if (lane == 0) {
      // ---- scales and MMAs ----
      int piece = -1;
      bool fresh = true;
      GWalk w(P);
      for (int i = 0, sl = 0, ph = 0; i < n; ++i, w.next()) {
        const int ks = w.ks;
        if (i == 0 || ks == 0) {             // a new tile: its accumulator is free?
          ++piece;
          fresh = true;
          if (piece >= S::kNacc &&
              !g_wait(&s_tempty[piece % S::kNacc], (uint32_t)((piece / S::kNacc) - 1) & 1u, &s_abort, a.status, 61))
            break;
          g_after();
        }
        if (!g_wait(&s_full[sl], (uint32_t)ph, &s_abort, a.status, 62)) break;
        g_after();
        const uint32_t st = base + (uint32_t)(sl * S::kStage);
        const uint32_t acc = tmem + (uint32_t)((piece % S::kNacc) * S::kAcc);
        const uint32_t sfa = tmem + (uint32_t)(S::kNacc * S::kAcc + sl * S::kSfCols);
        const uint32_t sfb = sfa + S::kAtoms * 4;
#pragma unroll
        for (int t = 0; t < S::kAtoms; ++t) {
          g_cp_sf(sfa + t * 4, g_desc(st + kGABytes + S::kB + t * kSfTile, 128, 0));
          g_cp_sf(sfb + t * 4, g_desc(st + kGABytes + S::kB + S::kSfA + t * kSfTile, 128, 0));
        }
        const int rest = a.d_in - ks * kGK;                    // inputs from this step on
#pragma unroll
        for (int kk = 0; kk < kGK / 64; ++kk) {
          if (kk * 64 < rest) {
            const uint64_t ad = g_desc(st + kk * 32, 1024, 2);
            const uint64_t bd = g_desc(st + kGABytes + kk * 32, 1024, 2);
            const int t = NV ? kk : kk >> 1;
            const uint32_t id = NV ? 0u : (uint32_t)(kk & 1) * 2u;
            g_mma<NV>(acc, ad, bd, g_idesc<NV, NT>(id), sfa + t * 4, sfb + t * 4, fresh ? 0u : 1u);
            fresh = false;
          }
        }
        g_commit(&s_empty[sl]);
        if (ks == nk - 1 || i == n - 1) g_commit(&s_tfull[piece % S::kNacc]);
        if (++sl == S::kStages) sl = 0, ph ^= 1;
      }
      g_commit(&s_done);                    // every MMA issued has completed when this arrives
      mbar_wait(&s_done, 0u);
    }
  } else {
    // ---- results ----
    asm volatile("griddepcontrol.wait;" ::: "memory");         // the tensor scale, and y's last readers
    const int q = warp & 3;
    if (NV) scale = __fmul_rn(a.x_scale ? *(volatile const float*)a.x_scale : 1.0f,
                              a.w_scale ? *(volatile const float*)a.w_scale : 1.0f);
    int piece = 0;
    GWalk w(P);
    for (int left = n; left > 0; ++piece) {
      const int len = gmin(left, nk - w.ks);
      const int col = w.mt * kGM + q * 32 + lane;
      const int tok0 = w.nt * NT, ntok = gmin(NT, a.T - tok0);
      const bool ok = g_wait_warp(&s_tfull[piece % S::kNacc], (uint32_t)(piece / S::kNacc) & 1u, &s_abort, a.status, 63);
      g_after();
      const uint32_t acc = tmem + ((uint32_t)(q * 32) << 16) + (uint32_t)((piece % S::kNacc) * S::kAcc);
      // a shared tile's partial sums: [token][output] in the ring, which every
      // MMA has read by now
      const uint32_t part = base + (uint32_t)((q * 32 + lane) * 4);
#pragma unroll 1
      for (int c = 0; c < ntok && ok; c += 8) {
        uint32_t v[8];
        g_ld8(acc + (uint32_t)c, v);
        g_ld_wait();
        if (C == 1) {
          if (col < a.d_out) {
#pragma unroll
            for (int e = 0; e < 8; ++e) {
              if (c + e < ntok) g_store(a, (size_t)(tok0 + c + e) * a.d_out + col, __uint_as_float(v[e]), NV, scale);
            }
          }
        } else {
#pragma unroll
          for (int e = 0; e < 8; ++e)
            if (c + e < ntok)
              asm volatile("st.shared.u32 [%0], %1;" ::"r"(part + (uint32_t)((c + e) * kGM * 4)), "r"(v[e]) : "memory");
        }
      }
      g_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(&s_tempty[piece % S::kNacc]);
      left -= len;
      w.ks = nk - 1;
      w.next();
    }
  }
  if (C > 1) {
    // every thread of the cluster reaches both barriers
    asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::: "memory");
    if (warp >= 2) {
      const GWalk w(P);
      const int tok0 = w.nt * NT, ntok = gmin(NT, a.T - tok0);
      const int items = ntok * (kGM / 4);
      for (int i = rank * 128 + (int)threadIdx.x - 64; i < items; i += C * 128) {
        const int t = i / (kGM / 4), c = (i % (kGM / 4)) * 4, col = w.mt * kGM + c;
        if (col >= a.d_out) continue;               // d_out is a multiple of 8
        const uint32_t local = base + (uint32_t)((t * kGM + c) * 4);
        float sum[4] = {0.0f, 0.0f, 0.0f, 0.0f};
        for (int r = 0; r < C; ++r) {
          uint32_t remote;
          float v[4];
          asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(remote) : "r"(local), "r"(r));
          asm volatile("ld.shared::cluster.v4.f32 {%0, %1, %2, %3}, [%4];"
                       : "=f"(v[0]), "=f"(v[1]), "=f"(v[2]), "=f"(v[3])
                       : "r"(remote)
                       : "memory");
#pragma unroll
          for (int e = 0; e < 4; ++e) sum[e] += v[e];
        }
#pragma unroll
        for (int e = 0; e < 4; ++e) g_store(a, (size_t)(tok0 + t) * a.d_out + col + e, sum[e], NV, scale);
      }
    }
    // no CTA leaves while another may still read its shared memory
    asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::: "memory");
  }
  g_before();
  __syncthreads();
  if (warp == 1) {
    g_after();
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(512u) : "memory");
  }
}

template <bool NV, int NT>
cudaError_t g_launch(const CUtensorMap& mw, const CUtensorMap& mx, const Fp4GemmArgs& a, cudaStream_t s) {
  static unsigned configured = 0;
  cudaError_t e = ensure_smem_attr(fp4_gemm_kernel<NV, NT>, GShape<NV, NT>::kSmem, &configured);
  if (e != cudaSuccess) return e;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)a.plan.grid);
  cfg.blockDim = dim3(kGThreads);
  cfg.dynamicSmemBytes = (size_t)GShape<NV, NT>::kSmem;
  cfg.stream = s;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = (unsigned)a.plan.cluster;
  attr[1].val.clusterDim.y = 1;
  attr[1].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 2;
  e = cudaLaunchKernelEx(&cfg, fp4_gemm_kernel<NV, NT>, mw, mx, a);
  if (e != cudaSuccess) return e;
  return cudaGetLastError();
}

// Clusters of c CTAs that are resident at once (one CTA per SM; every instance
// takes most of an SM's shared memory, so one of them answers for all).
int g_max_clusters(int c) {
  static std::once_flag once;
  static int n[9] = {0};
  std::call_once(once, [] {
    auto k = fp4_gemm_kernel<true, 128>;
    constexpr int smem = GShape<true, 128>::kSmem;
    static_assert(smem > 114 * 1024, "one CTA per SM");
    if (cudaFuncSetAttribute(k, cudaFuncAttributeMaxDynamicSharedMemorySize, smem) != cudaSuccess) {
      (void)cudaGetLastError();
      return;
    }
    for (int i = 1; i <= 8; ++i) {
      cudaLaunchConfig_t cfg = {};
      cfg.gridDim = dim3((unsigned)(i * kNumSMs));
      cfg.blockDim = dim3(kGThreads);
      cfg.dynamicSmemBytes = smem;
      cudaLaunchAttribute attr[1];
      attr[0].id = cudaLaunchAttributeClusterDimension;
      attr[0].val.clusterDim.x = (unsigned)i;
      attr[0].val.clusterDim.y = 1;
      attr[0].val.clusterDim.z = 1;
      cfg.attrs = attr;
      cfg.numAttrs = 1;
      int m = 0;
      if (cudaOccupancyMaxActiveClusters(&m, k, &cfg) == cudaSuccess) n[i] = m;
      (void)cudaGetLastError();
    }
  });
  return n[c];
}

template <bool NV>
cudaError_t g_dispatch(const CUtensorMap& mw, const CUtensorMap& mx, const Fp4GemmArgs& a, cudaStream_t s) {
  switch (a.plan.nt) {
    case 8: return g_launch<NV, 8>(mw, mx, a, s);
    case 16: return g_launch<NV, 16>(mw, mx, a, s);
    case 32: return g_launch<NV, 32>(mw, mx, a, s);
    case 64: return g_launch<NV, 64>(mw, mx, a, s);
    case 128: return g_launch<NV, 128>(mw, mx, a, s);
    default: return cudaErrorInvalidValue;
  }
}

}  // namespace

bool fp4_gemm_supported() { return g_encode_fn() != nullptr; }

Fp4GemmPlan plan_fp4_gemm(int T, int d_in, int d_out) {
  Fp4GemmPlan p;
  p.mtiles = (d_out + kGM - 1) / kGM;
  p.nk = (d_in + kGK - 1) / kGK;
  // tiles of 256 x 256 on two SMs where they give every pair one, else the
  // smallest tile of 128 outputs that holds the tokens (at most 128)
  if (T > 128 && fp4_wide_pairs() > 0 && (long)((T + 255) / 256) * ((d_out + 255) / 256) >= fp4_wide_pairs()) {
    p.nt = 256;
    return p;
  }
  p.nt = 8;
  while (p.nt < T && p.nt < 128) p.nt *= 2;
  p.ntiles = (T + p.nt - 1) / p.nt;
  const long tiles = (long)p.mtiles * p.ntiles;
  // the largest cluster of which every tile has one at once, with at least 2
  // steps per CTA (a step is less than the hand-over costs)
  p.cluster = 1;
  for (int c = 2; c <= 8 && 2 * c <= p.nk; ++c)
    if (tiles <= g_max_clusters(c)) p.cluster = c;
  p.grid = p.cluster > 1 ? (int)tiles * p.cluster : (int)(tiles < kNumSMs ? tiles : kNumSMs);
  return p;
}

cudaError_t launch_fp4_gemm(const Fp4GemmArgs& a, cudaStream_t s) {
  if (a.plan.nt == 256) return launch_fp4_gemm_wide(a, s);
  CUtensorMap mw, mx;
  if (!g_map(&mw, a.wc, (uint64_t)(a.d_in / 2), (uint64_t)a.d_out, kGM) ||
      !g_map(&mx, a.xc, (uint64_t)(a.d_in / 2), (uint64_t)a.T, (uint32_t)a.plan.nt))
    return cudaErrorInvalidValue;
  return a.format == QS_FP4_NV ? g_dispatch<true>(mw, mx, a, s) : g_dispatch<false>(mw, mx, a, s);
}

}  // namespace qs
