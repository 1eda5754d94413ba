// Quantisation of rows to microscaled 4-bit floating point.
//
//   MX: block of 32, s = 2^(floor(log2 amax) - 2) (e8m0), q = e2m1(x / s)
//   NV: block of 16, s = e4m3((amax / 6) / g), r = s * g, q = e2m1(x * (1 / r))
// in float32 steps, each rounded to nearest even; q saturates at 6 (a block's
// largest value lies in [4, 8) s for MX).  The reciprocal of r is taken once a
// block, so that a value costs one product.
//
// Bound by memory: 2 or 4 bytes read and 0.53 or 0.56 written per value (plus
// the rounded values, where asked for).  A thread takes 8 neighbouring values
// (one 16-byte load of bf16, two of f32), the 4 or 2 threads of a block share
// its largest magnitude by shuffles, and the codes leave as one 32-bit word
// per thread, so that loads and stores are whole 128-byte lines without
// staging in shared memory.
#include "fp4.cuh"

namespace qs {
namespace {

constexpr int kQThreads = 256;

// (volatile: not to be moved above the wait for the kernel that wrote x)
__device__ __forceinline__ uint4 ld_x(const void* p) {
  uint4 r;
  asm volatile("ld.global.nc.L1::no_allocate.v4.u32 {%0,%1,%2,%3}, [%4];"
               : "=r"(r.x), "=r"(r.y), "=r"(r.z), "=r"(r.w)
               : "l"(p));
  return r;
}

template <bool BF16>
__device__ __forceinline__ void load8(const void* x, size_t v, float (&f)[8]) {
  if constexpr (BF16) {
    const uint4 u = ld_x(reinterpret_cast<const uint4*>(x) + v);
    const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      f[2 * i] = bf16lo(w[i]);
      f[2 * i + 1] = bf16hi(w[i]);
    }
  } else {
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const uint4 u = ld_x(reinterpret_cast<const uint4*>(x) + 2 * v + i);
      f[4 * i] = __uint_as_float(u.x);
      f[4 * i + 1] = __uint_as_float(u.y);
      f[4 * i + 2] = __uint_as_float(u.z);
      f[4 * i + 3] = __uint_as_float(u.w);
    }
  }
}

template <bool BF16, bool NV>
__device__ __forceinline__ void quant8(const Fp4QuantArgs& a, size_t v, const float (&f)[8], float g,
                                       bool small) {
  // the block's largest magnitude, as bits (non-finite values rank above all
  // finite ones); the threads of a block are neighbours in one warp
  uint32_t m = 0;
#pragma unroll
  for (int i = 0; i < 8; ++i) m = max(m, __float_as_uint(f[i]) & 0x7fffffffu);
  m = max(m, __shfl_xor_sync(0xffffffffu, m, 1));
  if constexpr (!NV) m = max(m, __shfl_xor_sync(0xffffffffu, m, 2));
  const bool finite = m < 0x7f800000u;
  uint32_t code;                    // the block's scale byte
  float inv, back;                  // x * inv is what e2m1 rounds; back takes it to x's units
  if constexpr (NV) {
    const float amax = __uint_as_float(m);
    const float t = __fdiv_rn(__fdiv_rn(amax, 6.0f), g);
    const __nv_fp8_storage_t s8 = __nv_cvt_float_to_fp8(t, __NV_SATFINITE, __NV_E4M3);
    code = finite ? (uint32_t)s8 : 0x7fu;
    const float s = __half2float(__half(__nv_cvt_fp8_to_halfraw(s8, __NV_E4M3)));
    back = __fmul_rn(s, g);
    // below the smallest normal number the reciprocal would overflow: such a
    // block becomes 0
    inv = back >= 1.17549435e-38f ? __fdiv_rn(1.0f, back) : 0.0f;
  } else {
    const uint32_t be = m >> 23;    // biased exponent: floor(log2 amax) + 127 (0: below 2^-126)
    code = finite ? (be > 2u ? be - 2u : 0u) : 255u;
    inv = __uint_as_float((254u - code) << 23);          // 2^(127 - code)
    back = e8m0_value(code);
  }
  if (!finite) { inv = 0.0f; back = __uint_as_float(0x7fc00000u); }
  float q[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) q[i] = finite ? __fmul_rn(f[i], inv) : 0.0f;
  const uint32_t c = e2m1x8(q);
  if (a.codes) reinterpret_cast<uint32_t*>(a.codes)[v] = c;
  constexpr int kTpb = NV ? 2 : 4;  // threads per block
  if (a.scales && (threadIdx.x & (kTpb - 1)) == 0) {
    const size_t blk = v / kTpb;    // block number over all rows
    if (a.tiled) {
      const uint32_t nb = (uint32_t)(a.d / (8 * kTpb));
      size_t row, b;
      if (small) {
        row = (uint32_t)blk / nb;
        b = (uint32_t)blk - (uint32_t)row * nb;
      } else {
        row = blk / nb;
        b = blk - row * nb;
      }
      a.scales[fp4_tiled_offset(row, (int)b, fp4_tiles_per_row((int)nb))] = (uint8_t)code;
    } else {
      a.scales[blk] = (uint8_t)code;
    }
  }
  if (a.values) {
    uint32_t h[4];
    e2m1x8_to_half2(c, h);
    float o[8];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float2 p = __half22float2(*reinterpret_cast<const __half2*>(&h[i]));
      o[2 * i] = __fmul_rn(p.x, back);
      o[2 * i + 1] = __fmul_rn(p.y, back);
    }
    if constexpr (BF16) {
      uint32_t w[4];
#pragma unroll
      for (int i = 0; i < 4; ++i)
        w[i] = (uint32_t)f32_to_bf16_bits(o[2 * i]) | ((uint32_t)f32_to_bf16_bits(o[2 * i + 1]) << 16);
      reinterpret_cast<uint4*>(a.values)[v] = make_uint4(w[0], w[1], w[2], w[3]);
    } else {
      reinterpret_cast<float4*>(a.values)[2 * v] = make_float4(o[0], o[1], o[2], o[3]);
      reinterpret_cast<float4*>(a.values)[2 * v + 1] = make_float4(o[4], o[5], o[6], o[7]);
    }
  }
}

// U: vectors of 8 values a thread loads before it rounds the first
template <bool BF16, bool NV, int U>
__global__ void __launch_bounds__(kQThreads) fp4_quant_kernel(Fp4QuantArgs a) {
  pdl_begin();
  const size_t n8 = a.R * (size_t)(a.d / 8);           // a multiple of 4: blocks are whole
  const bool small = n8 < (1ull << 32);
  const float g = (NV && a.tensor_scale) ? *a.tensor_scale : 1.0f;
  const size_t step = (size_t)gridDim.x * kQThreads * U;
  for (size_t v0 = (size_t)blockIdx.x * kQThreads * U + threadIdx.x; v0 - threadIdx.x < n8; v0 += step) {
    float f[U][8];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const size_t v = v0 + (size_t)u * kQThreads;
      if (v < n8) {
        load8<BF16>(a.x, v, f[u]);
      } else {
#pragma unroll
        for (int i = 0; i < 8; ++i) f[u][i] = 0.0f;
      }
    }
#pragma unroll
    for (int u = 0; u < U; ++u) {
      // whole warps agree where n8 is a multiple of 32 vectors; elsewhere the
      // shuffles still need every lane, so the threads behind the end take
      // part with zeros (the threads of one block are on one side of the end)
      const size_t v = v0 + (size_t)u * kQThreads;
      if (v - (threadIdx.x & 31) < n8) {
        Fp4QuantArgs b = a;
        if (v >= n8) b.codes = nullptr, b.scales = nullptr, b.values = nullptr;
        quant8<BF16, NV>(b, v, f[u], g, small);
      }
    }
  }
  // tiled scales: the blocks that fill a row's last tile and the rows that
  // fill the last tile are 0 (the tensor core multiplies the former with zeros)
  if (a.scales && a.tiled) {
    const int nb = a.d / (NV ? 16 : 32);
    const size_t tpr = fp4_tiles_per_row(nb);
    const int rest = (int)(tpr * 4) - nb;
    const size_t tid = (size_t)blockIdx.x * kQThreads + threadIdx.x, nthr = (size_t)gridDim.x * kQThreads;
    for (size_t i = tid; i < a.R * (size_t)rest; i += nthr)
      a.scales[fp4_tiled_offset(i / rest, nb + (int)(i % rest), tpr)] = 0;
    if (a.pad_rows) {
      const size_t over = (a.R + 127) / 128 * 128 - a.R;
      for (size_t i = tid; i < over * tpr; i += nthr)
        *reinterpret_cast<uint32_t*>(a.scales + fp4_tiled_offset(a.R + i / tpr, (int)(i % tpr) * 4, tpr)) = 0u;
    }
  }
}

// ---- top-K and quantisation of a row in one kernel ------------------------------
// One CTA per row; a thread keeps NV vectors of 8 neighbouring values in registers
// (vector v of thread t: values (v * threads + t) * 8 ...), so that the row is
// read once and only its codes and scales are written.  The K-th largest |x| (as
// bits) is found by radix passes of 11, 10 and 10 bits (bf16: 11 and 4) on
// histograms in shared memory: 2048 bins spread the few exponents that a row's
// values share over enough addresses for the atomics.  Equal magnitudes at the
// threshold are kept in index order, by one scan, where not all of them are.
// Bound by latency for a few rows (the passes' barriers): with the masked row
// written and read again between two kernels a projection of one token 4096 -> 11008
// took 21 us, with this kernel 17.  Many rows are bound by instructions: 2048 rows
// of 4096 bf16 take 38 us (94 instructions a value; a list of the ties instead of scans
// and four bins per load: 41; 6 or 8 CTAs per SM instead of 4: 42).
template <int THREADS>
__device__ __forceinline__ int block_exclusive(int v, int* s_warp, int& total) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  int inc = v;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int u = __shfl_up_sync(0xffffffffu, inc, o);
    if (lane >= o) inc += u;
  }
  __syncthreads();
  if (lane == 31) s_warp[warp] = inc;
  __syncthreads();
  int before = 0;
  total = 0;
#pragma unroll
  for (int w = 0; w < THREADS / 32; ++w) {
    const int c = s_warp[w];
    if (w < warp) before += c;
    total += c;
  }
  return before + inc - v;
}

template <bool BF16, bool NV, int THREADS, int VECS>
__global__ void __launch_bounds__(THREADS) fp4_topk_quant_kernel(Fp4QuantArgs a) {
  constexpr int kBits = BF16 ? 15 : 31, kBins = 2048;
  __shared__ int s_hist[kBins];
  __shared__ int s_warp[THREADS / 32];
  __shared__ int s_digit, s_above, s_equal;
  const int tid = threadIdx.x, per = a.d / 8;
  pdl_begin();
  const float g = (NV && a.tensor_scale) ? *a.tensor_scale : 1.0f;
  const size_t row0 = (size_t)blockIdx.x * per;        // first vector of the row
  const bool small = row0 + per < (1ull << 32);
  float f[VECS][8];
#pragma unroll
  for (int v = 0; v < VECS; ++v) {
    const int at = v * THREADS + tid;
    if (at < per) {
      load8<BF16>(a.x, row0 + at, f[v]);
    } else {
#pragma unroll
      for (int i = 0; i < 8; ++i) f[v][i] = 0.0f;
    }
  }
  auto key_of = [&](float x) { return (__float_as_uint(x) & 0x7fffffffu) >> (BF16 ? 16 : 0); };

  // the threshold: digits from the top; `need` of the values that share the
  // digits so far are kept
  uint32_t prefix = 0;
  int shift = kBits, need = a.k, equal = 0;
  if (need > 0) {
#pragma unroll 1
    for (int pass = 0; shift > 0; ++pass) {
      const int bits = min(pass == 0 ? 11 : 10, shift);
      const uint32_t before = shift >= 31 ? 0u : prefix >> shift;     // digits so far
      shift -= bits;
      for (int i = tid; i < (1 << bits); i += THREADS) s_hist[i] = 0;
      __syncthreads();
#pragma unroll
      for (int v = 0; v < VECS; ++v) {
        if (v * THREADS + tid < per) {
#pragma unroll
          for (int i = 0; i < 8; ++i) {
            const uint32_t k = key_of(f[v][i]);
            if (pass == 0 || (k >> (shift + bits)) == before) atomicAdd(&s_hist[(k >> shift) & ((1u << bits) - 1u)], 1);
          }
        }
      }
      __syncthreads();
      // counts from the top: thread t has the bins of the t-th share from the top
      const int n = 1 << bits, share = (n + THREADS - 1) / THREADS;
      int mine = 0;
      for (int i = 0; i < share; ++i) {
        const int b = n - 1 - (tid * share + i);
        if (b >= 0) mine += s_hist[b];
      }
      int total;
      int above = block_exclusive<THREADS>(mine, s_warp, total);
      if (above < need && above + mine >= need) {
        for (int i = 0; i < share; ++i) {
          const int b = n - 1 - (tid * share + i), c = s_hist[b];
          if (above + c >= need) {
            s_digit = b;
            s_above = above;
            s_equal = c;
            break;
          }
          above += c;
        }
      }
      __syncthreads();
      prefix |= (uint32_t)s_digit << shift;
      need -= s_above;
      equal = s_equal;
      if (equal == need && shift > 0) break;           // every value that shares these digits is kept
      __syncthreads();
    }
  }
  const uint32_t low = prefix;                         // keys >= low are kept, or (ties) == low by index
  const bool ties = need > 0 && equal != need;
#pragma unroll
  for (int v = 0; v < VECS; ++v) {
    const int at = v * THREADS + tid;
    int rank = 0;
    if (ties) {
      int c = 0, total;
#pragma unroll
      for (int i = 0; i < 8; ++i) c += at < per && key_of(f[v][i]) == low;
      rank = block_exclusive<THREADS>(c, s_warp, total);
      // (need: what is left for this vector's round and those after it)
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const uint32_t k = key_of(f[v][i]);
        const bool keep = k > low || (k == low && rank < need);
        rank += k == low;
        if (!keep) f[v][i] = 0.0f;
      }
      need -= total;
    } else {
#pragma unroll
      for (int i = 0; i < 8; ++i)
        if (a.k == 0 || key_of(f[v][i]) < low) f[v][i] = 0.0f;
    }
    // (whole warps: a row is a multiple of 4 vectors, not of 32)
    if (at - (tid & 31) < per) {
      Fp4QuantArgs b = a;
      if (at >= per) b.codes = nullptr, b.scales = nullptr, b.values = nullptr;
      quant8<BF16, NV>(b, row0 + at, f[v], g, small);
    }
  }
  // the blocks that fill the row's last scale tile are 0
  const int nb = a.d / (NV ? 16 : 32);
  const size_t tpr = fp4_tiles_per_row(nb);
  for (int i = tid; i < (int)(tpr * 4) - nb; i += THREADS) a.scales[fp4_tiled_offset(blockIdx.x, nb + i, tpr)] = 0;
}

template <bool BF16, bool NV>
cudaError_t launch_topk_quant(const Fp4QuantArgs& a, cudaStream_t s) {
  const int per = a.d / 8;
  const dim3 grid((unsigned)a.R);
  // one vector per thread for a few rows (latency), two where rows queue for the
  // SMs, more for long rows
  if (per <= 128) return launch_pdl(fp4_topk_quant_kernel<BF16, NV, 128, 1>, grid, dim3(128), 0, s, a);
  if (per <= 256) return launch_pdl(fp4_topk_quant_kernel<BF16, NV, 256, 1>, grid, dim3(256), 0, s, a);
  if (per <= 512 && a.R > (size_t)kNumSMs * 2) return launch_pdl(fp4_topk_quant_kernel<BF16, NV, 256, 2>, grid, dim3(256), 0, s, a);
  if (per <= 512) return launch_pdl(fp4_topk_quant_kernel<BF16, NV, 512, 1>, grid, dim3(512), 0, s, a);
  if (per <= 1024) return launch_pdl(fp4_topk_quant_kernel<BF16, NV, 512, 2>, grid, dim3(512), 0, s, a);
  if (per <= 2048) return launch_pdl(fp4_topk_quant_kernel<BF16, NV, 1024, 2>, grid, dim3(1024), 0, s, a);
  return launch_pdl(fp4_topk_quant_kernel<BF16, NV, 1024, 6>, grid, dim3(1024), 0, s, a);
}

}  // namespace

cudaError_t launch_fp4_quantize(const Fp4QuantArgs& a, cudaStream_t s) {
  if (a.R == 0 || a.d <= 0) return cudaSuccess;
  const size_t n8 = a.R * (size_t)(a.d / 8);
  const bool nv = a.format == QS_FP4_NV;
  // four loads in flight per thread where every SM has its threads, else as
  // many threads as there are vectors (a few tokens: latency counts)
  const bool many = n8 > (size_t)kNumSMs * 8 * kQThreads;
  const size_t per = (size_t)kQThreads * (many ? 4 : 1);
  size_t grid = (n8 + per - 1) / per;
  if (grid > (size_t)kNumSMs * 8) grid = (size_t)kNumSMs * 8;
  void (*k)(Fp4QuantArgs);
  if (many)
    k = a.bf16 ? (nv ? fp4_quant_kernel<true, true, 4> : fp4_quant_kernel<true, false, 4>)
               : (nv ? fp4_quant_kernel<false, true, 4> : fp4_quant_kernel<false, false, 4>);
  else
    k = a.bf16 ? (nv ? fp4_quant_kernel<true, true, 1> : fp4_quant_kernel<true, false, 1>)
               : (nv ? fp4_quant_kernel<false, true, 1> : fp4_quant_kernel<false, false, 1>);
  cudaError_t e = launch_pdl(k, dim3((unsigned)grid), dim3(kQThreads), 0, s, a);
  if (e != cudaSuccess) return e;
  return cudaGetLastError();
}

cudaError_t launch_fp4_topk_quantize(const Fp4QuantArgs& a, cudaStream_t s) {
  const bool nv = a.format == QS_FP4_NV;
  const cudaError_t e = a.bf16 ? (nv ? launch_topk_quant<true, true>(a, s) : launch_topk_quant<true, false>(a, s))
                               : (nv ? launch_topk_quant<false, true>(a, s) : launch_topk_quant<false, false>(a, s));
  if (e != cudaSuccess) return e;
  return cudaGetLastError();
}

}  // namespace qs
