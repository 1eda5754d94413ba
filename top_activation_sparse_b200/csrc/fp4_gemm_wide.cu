// Product of two microscaled 4-bit matrices for many tokens: tiles of 256 tokens x
// 256 outputs, each on two SMs (tcgen05.mma.cta_group::2 with block scales).
//
// Same sum as fp4_gemm.cu.  With 4-bit operands a 128 x 256 tile on one SM asks
// L2 for 96 bytes per cycle and SM, more than it delivers (measured: 11 TB/s in
// all, about 42 bytes per cycle and SM), so a cluster of two CTAs shares a tile:
// each loads its own 128 tokens and its own half of the weight tile (38 KB per
// step of 256 inputs for 256 x 256 x 256, where two single tiles load 108 KB),
// and the tokens are the M side, so that a lane of an accumulator holds
// neighbouring outputs.
//   * each CTA's producer copies its codes (2-D TMA, 128-byte swizzle) and the
//     scales that its SM needs (its tokens' and all 256 outputs'; 2-D TMA over
//     the tiled layout, which fills what lies behind the last tile with zeros),
//     all signalling the first CTA's barrier;
//   * the first CTA's MMA thread copies the scales to both SMs' tensor memory
//     (tcgen05.cp, a place per ring stage) and issues the products;
//   * each CTA's epilogue warps round their 128 x 256 accumulator into shared
//     memory (swizzled), from where one thread stores it by TMA, which clips the
//     ragged edges; the accumulator is free again as soon as it has been read.
// 128 x 256 tiles with stores from registers: 130 us for 2048 tokens, 4096 ->
// 11008 (NV); this kernel 76 us, 2.4 PFLOP/s.  L2 delivers the operands in 38 us (418 MB at the rate
// above), beside which the products (24 us: the tensor pipe is active 29.5% of a profiled 80.8 us)
// and the copies of the scales to tensor memory (20 us; asking for them a step ahead: 95 us in
// all) run in turn; with one accumulator no product runs while a tile's results are
// read.  Every wait is bounded.
#include <mutex>

#include "fp4_mma.cuh"

namespace qs {
namespace {

constexpr int kWThreads = 192;
constexpr int kWK = 256;                       // inputs per step: 128 bytes of codes per row
constexpr int kWRows = 128;                    // rows of each operand per CTA
constexpr int kWOp = kWRows * kWK / 2;         // 16 KB
constexpr int kWStages = 4;
constexpr int kWOut = 64 * 1024;               // rounded results: four (bf16) or two halves of four (f32) 16 KB boxes

template <bool NV>
struct WShape {
  static constexpr int kAtoms = kWK / (NV ? 16 : 32) / 4;        // 512-byte scale tiles per step
  static constexpr int kSfA = kAtoms * kSfTile, kSfB = 2 * kSfA;
  static constexpr int kStage = 2 * kWOp + kSfA + kSfB;
  static constexpr int kSfCols = kAtoms * 4 * 3;                 // tensor-memory columns per stage
  static constexpr int kSmem = kWStages * kStage + kWOut + 1024;
  static_assert(256 + kWStages * kSfCols <= 512, "tensor memory");
  static_assert(kStage % 1024 == 0 && kSmem <= 226 * 1024, "shared memory");
};

// e2m1 x e2m1, K-major, f32, M = 256 (the pair), N = 256
template <bool NV>
__device__ constexpr uint32_t w_idesc(uint32_t sf_id) {
  return (sf_id << 4) | (1u << 7) | (1u << 10) | ((uint32_t)(256 >> 3) << 17) | ((NV ? 0u : 1u) << 23) |
         ((uint32_t)(256 >> 4) << 24) | (sf_id << 29);
}
template <bool NV>
__device__ __forceinline__ void w_mma(uint32_t d, uint64_t ad, uint64_t bd, uint32_t idesc, uint32_t sfa, uint32_t sfb,
                                      uint32_t accumulate) {
  if constexpr (NV)
    asm volatile(
        "{\n .reg .pred p;\n setp.ne.u32 p, %6, 0;\n"
        " tcgen05.mma.cta_group::2.kind::mxf4nvf4.block_scale.scale_vec::4X [%0], %1, %2, %3, [%4], [%5], p;\n}\n" ::"r"(d),
        "l"(ad), "l"(bd), "r"(idesc), "r"(sfa), "r"(sfb), "r"(accumulate)
        : "memory");
  else
    asm volatile(
        "{\n .reg .pred p;\n setp.ne.u32 p, %6, 0;\n"
        " tcgen05.mma.cta_group::2.kind::mxf4.block_scale.scale_vec::2X [%0], %1, %2, %3, [%4], [%5], p;\n}\n" ::"r"(d),
        "l"(ad), "l"(bd), "r"(idesc), "r"(sfa), "r"(sfb), "r"(accumulate)
        : "memory");
}
__device__ __forceinline__ void w_cp_sf(uint32_t taddr, uint64_t sdesc) {
  asm volatile("tcgen05.cp.cta_group::2.32x128b.warpx4 [%0], %1;" ::"r"(taddr), "l"(sdesc) : "memory");
}
// once the work issued so far has completed: the barrier at this offset in both CTAs
__device__ __forceinline__ void w_commit(uint64_t* bar) {
  const uint16_t mask = 0x3;
  asm volatile(
      "tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64 [%0], %1;" ::"r"(smem_u32(bar)),
      "h"(mask)
      : "memory");
}
__device__ __forceinline__ void w_commit_here(uint64_t* bar) {
  asm volatile("tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.b64 [%0];" ::"r"(smem_u32(bar)) : "memory");
}
__device__ __forceinline__ uint32_t w_peer(uint32_t local, uint32_t rank) {
  uint32_t r;
  asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(r) : "r"(local), "r"(rank));
  return r;
}
__device__ __forceinline__ void w_load(uint32_t dst, const CUtensorMap* map, int x, int y, uint32_t bar_cluster) {
  asm volatile(
      "cp.async.bulk.tensor.2d.cta_group::2.shared::cluster.global.mbarrier::complete_tx::bytes"
      " [%0], [%1, {%2, %3}], [%4];" ::"r"(dst),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(x), "r"(y), "r"(bar_cluster)
      : "memory");
}
__device__ __forceinline__ void w_store(const CUtensorMap* map, int x, int y, uint32_t src) {
  asm volatile("cp.async.bulk.tensor.2d.global.shared::cta.bulk_group [%0, {%1, %2}], [%3];" ::"l"(
                   reinterpret_cast<uint64_t>(map)),
               "r"(x), "r"(y), "r"(src)
               : "memory");
}
__device__ __forceinline__ void w_ld32(uint32_t taddr, uint32_t (&r)[32]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x32.b32 {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, "
      "%16, %17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31}, [%32];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]),
        "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15]), "=r"(r[16]), "=r"(r[17]),
        "=r"(r[18]), "=r"(r[19]), "=r"(r[20]), "=r"(r[21]), "=r"(r[22]), "=r"(r[23]), "=r"(r[24]), "=r"(r[25]), "=r"(r[26]),
        "=r"(r[27]), "=r"(r[28]), "=r"(r[29]), "=r"(r[30]), "=r"(r[31])
      : "r"(taddr));
  asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory");
}
__device__ __forceinline__ void w_cluster_sync() {
  asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::: "memory");
}
struct WMaps {
  CUtensorMap xc, wc, xs, ws, y;
};

template <bool NV, bool BF16>
__global__ void __launch_bounds__(kWThreads, 1) fp4_gemm_wide_kernel(const __grid_constant__ WMaps maps, Fp4GemmArgs a) {
  using S = WShape<NV>;
  extern __shared__ __align__(1024) unsigned char smem_raw[];
  __shared__ __align__(8) uint64_t s_full[kWStages];    // first CTA: both CTAs' copies of a stage
  __shared__ __align__(8) uint64_t s_empty[kWStages];   // each CTA: the stage's products are done
  __shared__ __align__(8) uint64_t s_tfull;             // each CTA: the accumulator is complete
  __shared__ __align__(8) uint64_t s_tempty;            // first CTA: both epilogues have read it
  __shared__ __align__(8) uint64_t s_done;
  __shared__ uint32_t s_tmem;
  __shared__ int s_abort;

  const uint32_t base = (smem_u32(smem_raw) + 1023u) & ~1023u;
  const uint32_t out = base + (uint32_t)(kWStages * S::kStage);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const uint32_t rank = blockIdx.x & 1u;
  const bool leader = rank == 0;
  const int pair = blockIdx.x >> 1, npairs = gridDim.x >> 1;
  const int mtiles = (a.T + 255) / 256, tiles = mtiles * ((a.d_out + 255) / 256);
  const int nk = (a.d_in + kWK - 1) / kWK;
  const int mine = pair < tiles ? (tiles - 1 - pair) / npairs + 1 : 0;

  if (threadIdx.x == 0) {
    for (int i = 0; i < kWStages; ++i) {
      mbar_init(&s_full[i], 1);
      mbar_init(&s_empty[i], 1);
    }
    mbar_init(&s_tfull, 1);
    mbar_init(&s_tempty, 8);
    mbar_init(&s_done, 1);
    mbar_fence_init();
    s_abort = 0;
  }
  if (warp == 0) {
    asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_u32(&s_tmem)), "r"(512u)
                 : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;" ::: "memory");
  }
  g_before();
  __syncthreads();
  w_cluster_sync();                                // the peer's barriers exist before any signal
  g_after();
  const uint32_t tmem = s_tmem;
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");

  if (warp == 0) {
    if (lane == 0) {
      // ---- copies (both CTAs) ----
      // the weights and their scales do not depend on the kernel that quantises
      // x: those of the first steps are asked for before waiting for it
      auto place = [&](int it, int& kb, int& m0, int& n0) {
        const int lt = it / nk, t = pair + lt * npairs;
        kb = it - lt * nk;
        m0 = (t % mtiles) * 256;
        n0 = (t / mtiles) * 256;
      };
      auto copy_w = [&](int it, int s) {
        int kb, m0, n0;
        place(it, kb, m0, n0);
        const uint32_t st = base + (uint32_t)(s * S::kStage), full = w_peer(smem_u32(&s_full[s]), 0);
        if (leader) mbar_arrive_expect_tx(&s_full[s], (uint32_t)(2 * S::kStage));
        w_load(st + kWOp, &maps.wc, kb * (kWK / 2), n0 + (int)rank * kWRows, full);
        w_load(st + 2 * kWOp + S::kSfA, &maps.ws, kb * S::kAtoms * 64, n0 / 128, full);
      };
      auto copy_x = [&](int it, int s) {
        int kb, m0, n0;
        place(it, kb, m0, n0);
        const uint32_t st = base + (uint32_t)(s * S::kStage), full = w_peer(smem_u32(&s_full[s]), 0);
        w_load(st, &maps.xc, kb * (kWK / 2), m0 + (int)rank * kWRows, full);
        w_load(st + 2 * kWOp, &maps.xs, kb * S::kAtoms * 64, m0 / 128 + (int)rank, full);
      };
      const int n = mine * nk, head = n < kWStages ? n : kWStages;
      for (int i = 0; i < head; ++i) copy_w(i, i);
      asm volatile("griddepcontrol.wait;" ::: "memory");
      for (int i = 0; i < head; ++i) copy_x(i, i);
      int it = head;
      for (; it < n; ++it) {
        const int s = it % kWStages;
        if (!g_wait(&s_empty[s], (uint32_t)((it / kWStages) - 1) & 1u, &s_abort, a.status, 90)) break;
        copy_w(it, s);
        copy_x(it, s);
      }
      // after a give-up the first CTA lets the copies in flight (both CTAs') land
      if (leader && *(volatile int*)&s_abort)
        for (int j = 0; j < kWStages && j < it; ++j) {
          const int g = it - 1 - j;
          mbar_wait(&s_full[g % kWStages], (uint32_t)(g / kWStages) & 1u);
        }
    }
  } else if (warp == 1) {
    if (lane == 0 && leader) {
      // ---- scales and products (first CTA) ----
      int it = 0;
      bool issued = false, ok = true;
      for (int lt = 0; lt < mine && ok; ++lt) {
        if (lt >= 1 && !g_wait(&s_tempty, (uint32_t)(lt - 1) & 1u, &s_abort, a.status, 91)) break;
        g_after();
        for (int kb = 0; kb < nk; ++kb, ++it) {
          const int s = it % kWStages;
          if (!g_wait(&s_full[s], (uint32_t)(it / kWStages) & 1u, &s_abort, a.status, 92)) {
            ok = false;
            break;
          }
          g_after();
          const uint32_t st = base + (uint32_t)(s * S::kStage);
          const uint32_t sfa = tmem + 256u + (uint32_t)(s * S::kSfCols), sfb = sfa + S::kAtoms * 4;
#pragma unroll
          for (int t = 0; t < S::kAtoms; ++t) {
            w_cp_sf(sfa + t * 4, g_desc(st + 2 * kWOp + t * kSfTile, 128, 0));
#pragma unroll
            for (int r = 0; r < 2; ++r)
              w_cp_sf(sfb + (t * 2 + r) * 4, g_desc(st + 2 * kWOp + S::kSfA + (r * S::kAtoms + t) * kSfTile, 128, 0));
          }
          const int rest = a.d_in - kb * kWK;
#pragma unroll
          for (int kk = 0; kk < kWK / 64; ++kk) {
            if (kk * 64 < rest) {
              const int t = NV ? kk : kk >> 1;
              const uint32_t id = NV ? 0u : (uint32_t)(kk & 1) * 2u;
              w_mma<NV>(tmem, g_desc(st + kk * 32, 1024, 2), g_desc(st + kWOp + kk * 32, 1024, 2), w_idesc<NV>(id), sfa + t * 4,
                        sfb + t * 8, (kb > 0 || kk > 0) ? 1u : 0u);
            }
          }
          w_commit(&s_empty[s]);                   // frees the stage in both CTAs
          issued = true;
        }
        w_commit(&s_tfull);
      }
      if (issued) {
        w_commit_here(&s_done);
        mbar_wait(&s_done, 0u);
      }
    }
  } else {
    // ---- results (both CTAs): this CTA's 128 tokens ----
    asm volatile("griddepcontrol.wait;" ::: "memory");
    const int q = warp & 3;
    float scale = 1.0f;
    if (NV) scale = __fmul_rn(a.x_scale ? *(volatile const float*)a.x_scale : 1.0f, a.w_scale ? *(volatile const float*)a.w_scale : 1.0f);
    const uint32_t tempty0 = w_peer(smem_u32(&s_tempty), 0);
    const int row = q * 32 + lane;
    constexpr int kBoxCols = BF16 ? 64 : 32;       // 128 bytes
    for (int lt = 0; lt < mine; ++lt) {
      const int t = pair + lt * npairs;
      const int m0 = (t % mtiles) * 256 + (int)rank * kWRows, n0 = (t / mtiles) * 256;
      const bool ok = g_wait_warp(&s_tfull, (uint32_t)lt & 1u, &s_abort, a.status, 93);
      g_after();
#pragma unroll
      for (int half = 0; half < (BF16 ? 1 : 2); ++half) {
        // the stores of the results before have read the shared memory
        if (threadIdx.x == 64) asm volatile("cp.async.bulk.wait_group.read 0;" ::: "memory");
        asm volatile("bar.sync 1, 128;" ::: "memory");
        constexpr int kCols = BF16 ? 256 : 128;
#pragma unroll 1
        for (int c = 0; c < kCols; c += 32) {
          uint32_t v[32];
          w_ld32(tmem + ((uint32_t)(q * 32) << 16) + (uint32_t)(half * 128 + c), v);
#pragma unroll
          for (int e = 0; e < 32; ++e) v[e] = NV ? __float_as_uint(__fmul_rn(__uint_as_float(v[e]), scale)) : v[e];
          // 16-byte chunk k of row r of a box lies at k ^ (r % 8)
          const uint32_t box = out + (uint32_t)(c / kBoxCols * 16384 + row * 128);
          if constexpr (BF16) {
#pragma unroll
            for (int k = 0; k < 4; ++k) {
              uint32_t p[4];
#pragma unroll
              for (int e = 0; e < 4; ++e)
                p[e] = (uint32_t)f32_to_bf16_bits(__uint_as_float(v[8 * k + 2 * e])) |
                       ((uint32_t)f32_to_bf16_bits(__uint_as_float(v[8 * k + 2 * e + 1])) << 16);
              const uint32_t to = box + (uint32_t)((((c % 64) / 8 + k) ^ (row & 7)) * 16);
              asm volatile("st.shared.v4.u32 [%0], {%1, %2, %3, %4};" ::"r"(to), "r"(p[0]), "r"(p[1]), "r"(p[2]), "r"(p[3]) : "memory");
            }
          } else {
#pragma unroll
            for (int k = 0; k < 8; ++k) {
              const uint32_t to = box + (uint32_t)((k ^ (row & 7)) * 16);
              asm volatile("st.shared.v4.u32 [%0], {%1, %2, %3, %4};" ::"r"(to), "r"(v[4 * k]), "r"(v[4 * k + 1]), "r"(v[4 * k + 2]),
                           "r"(v[4 * k + 3])
                           : "memory");
            }
          }
        }
        if (half == (BF16 ? 0 : 1)) {
          g_before();
          __syncwarp();
          if (lane == 0)
            asm volatile("mbarrier.arrive.release.cluster.shared::cluster.b64 _, [%0];" ::"r"(tempty0) : "memory");
        }
        asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
        asm volatile("bar.sync 1, 128;" ::: "memory");
        if (threadIdx.x == 64 && ok && !*(volatile int*)&s_abort) {
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            const int x = n0 + half * 128 + k * kBoxCols;
            if (x < a.d_out && m0 < a.T) w_store(&maps.y, x, m0, out + (uint32_t)(k * 16384));
          }
          asm volatile("cp.async.bulk.commit_group;" ::: "memory");
        }
      }
    }
    if (threadIdx.x == 64) asm volatile("cp.async.bulk.wait_group 0;" ::: "memory");
  }
  g_before();
  __syncthreads();
  w_cluster_sync();                                // both CTAs are done with the pair's tensor memory
  if (warp == 0) {
    g_after();
    asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(512u) : "memory");
  }
}

bool w_map(CUtensorMap* m, CUtensorMapDataType dt, const void* ptr, uint64_t inner, uint64_t outer, uint64_t pitch, uint32_t bx,
           uint32_t by, bool swizzle) {
  auto fn = g_encode_fn();
  if (fn == nullptr) return false;
  cuuint64_t dims[2] = {inner, outer};
  cuuint64_t strides[1] = {pitch};
  cuuint32_t box[2] = {bx, by};
  cuuint32_t estr[2] = {1, 1};
  return fn(m, dt, 2, const_cast<void*>(ptr), dims, strides, box, estr, CU_TENSOR_MAP_INTERLEAVE_NONE,
            swizzle ? CU_TENSOR_MAP_SWIZZLE_128B : CU_TENSOR_MAP_SWIZZLE_NONE, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
            CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

template <bool NV, bool BF16>
cudaError_t w_launch(const WMaps& maps, const Fp4GemmArgs& a, int pairs, cudaStream_t s) {
  static unsigned configured = 0;
  cudaError_t e = ensure_smem_attr(fp4_gemm_wide_kernel<NV, BF16>, WShape<NV>::kSmem, &configured);
  if (e != cudaSuccess) return e;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)(2 * pairs));
  cfg.blockDim = dim3(kWThreads);
  cfg.dynamicSmemBytes = (size_t)WShape<NV>::kSmem;
  cfg.stream = s;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = 2;
  attr[0].val.clusterDim.y = 1;
  attr[0].val.clusterDim.z = 1;
  attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[1].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 2;
  e = cudaLaunchKernelEx(&cfg, fp4_gemm_wide_kernel<NV, BF16>, maps, a);
  if (e != cudaSuccess) return e;
  return cudaGetLastError();
}

}  // namespace

// Pairs of SMs that are resident at once (0: not available; every instance
// takes most of an SM's shared memory, so one of them answers for all).
int fp4_wide_pairs() {
  static std::once_flag once;
  static int n = 0;
  std::call_once(once, [] {
    auto k = fp4_gemm_wide_kernel<true, true>;
    constexpr int smem = WShape<true>::kSmem;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(2 * kNumSMs);
    cfg.blockDim = dim3(kWThreads);
    cfg.dynamicSmemBytes = smem;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = 2;
    attr[0].val.clusterDim.y = 1;
    attr[0].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    int c = 0;
    if (cudaFuncSetAttribute(k, cudaFuncAttributeMaxDynamicSharedMemorySize, smem) == cudaSuccess &&
        cudaOccupancyMaxActiveClusters(&c, k, &cfg) == cudaSuccess)
      n = c;
    (void)cudaGetLastError();
  });
  return n;
}

cudaError_t launch_fp4_gemm_wide(const Fp4GemmArgs& a, cudaStream_t s) {
  const bool nv = a.format == QS_FP4_NV;
  const uint64_t tpr = fp4_tiles_per_row(a.d_in / fp4_block(a.format));
  const uint32_t sf_box = (uint32_t)(kWK / fp4_block(a.format) / 4 * 64);     // 8-byte elements per step
  WMaps m;
  if (!w_map(&m.xc, CU_TENSOR_MAP_DATA_TYPE_UINT8, a.xc, (uint64_t)(a.d_in / 2), (uint64_t)a.T, (uint64_t)(a.d_in / 2), kWK / 2, kWRows,
             true) ||
      !w_map(&m.wc, CU_TENSOR_MAP_DATA_TYPE_UINT8, a.wc, (uint64_t)(a.d_in / 2), (uint64_t)a.d_out, (uint64_t)(a.d_in / 2), kWK / 2,
             kWRows, true) ||
      !w_map(&m.xs, CU_TENSOR_MAP_DATA_TYPE_UINT64, a.xs, tpr * 64, (uint64_t)((a.T + 127) / 128), tpr * 512, sf_box, 1, false) ||
      !w_map(&m.ws, CU_TENSOR_MAP_DATA_TYPE_UINT64, a.ws, tpr * 64, (uint64_t)((a.d_out + 127) / 128), tpr * 512, sf_box, 2, false) ||
      !w_map(&m.y, a.y_bf16 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_FLOAT32, a.y, (uint64_t)a.d_out,
             (uint64_t)a.T, (uint64_t)a.d_out * (a.y_bf16 ? 2 : 4), a.y_bf16 ? 64 : 32, kWRows, true))
    return cudaErrorInvalidValue;
  const int tiles = ((a.T + 255) / 256) * ((a.d_out + 255) / 256), most = fp4_wide_pairs();
  const int pairs = tiles < most ? tiles : most;
  if (pairs < 1) return cudaErrorInvalidConfiguration;
  if (nv) return a.y_bf16 ? w_launch<true, true>(m, a, pairs, s) : w_launch<true, false>(m, a, pairs, s);
  return a.y_bf16 ? w_launch<false, true>(m, a, pairs, s) : w_launch<false, false>(m, a, pairs, s);
}

}  // namespace qs
