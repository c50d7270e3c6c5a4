// Quantisation to E4M3 codes with one fp32 scale per block of 128: activations by rows
// (a scale per 1 x 128 group) and weights by squares (a scale per 128 x 128 block).
//
//   scale  = amax(|x|) / 448                  (one fp32 division; 448 is the largest E4M3 value)
//   code_i = E4M3_rn_sat(x_i / scale)         (one fp32 division); 0 where scale == 0
//
// A NaN in a block makes its scale and all its codes NaN; an infinity makes the scale infinite,
// its own code NaN and the finite codes 0.
//
// Both are one pass over the input: a block is held in registers between its maximum and its
// codes. Element bytes + 1 per element: 8192 x 2688 bf16 takes 14.2 us (4.7 TB/s; 23.1 with IEEE
// divisions), 8192 x 14336 64 us (5.5 TB/s), weights of 14336 x 4096 bf16 36.7 us (4.8 TB/s), fp32
// 52.5 us (5.6 TB/s). The launch bounds keep as many CTAs on an SM as their registers allow, since
// each CTA's loads and stores alternate.
#include <cstdint>

#include "common.cuh"
#include "internal.h"

namespace fi {

namespace {

// Two fp32 values to two E4M3 codes (low byte = lo), round to nearest even, saturating.
__device__ __forceinline__ uint32_t f32x2_to_e4m3x2(float lo, float hi) {
  unsigned short r;
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(r) : "f"(hi), "f"(lo));
  return r;
}

// 16 bytes of input (DT = fi_dtype): as fp32, and the greatest magnitude in them.
template <int DT>
struct Vec;
template <>
struct Vec<FI_DTYPE_F32> {
  static constexpr int kN = 4;
  __device__ static void unpack(const uint4 v, float* x) {
    x[0] = __uint_as_float(v.x);
    x[1] = __uint_as_float(v.y);
    x[2] = __uint_as_float(v.z);
    x[3] = __uint_as_float(v.w);
  }
  __device__ static float amax(const uint4 v) {
    return max_nan(max_nan(fabsf(__uint_as_float(v.x)), fabsf(__uint_as_float(v.y))),
                   max_nan(fabsf(__uint_as_float(v.z)), fabsf(__uint_as_float(v.w))));
  }
};
template <>
struct Vec<FI_DTYPE_BF16> {
  static constexpr int kN = 8;
  __device__ static void unpack(const uint4 v, float* x) {
    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (int q = 0; q < 4; ++q) {
      x[2 * q] = __uint_as_float(w[q] << 16);
      x[2 * q + 1] = __uint_as_float(w[q] & 0xFFFF0000u);
    }
  }
  __device__ static uint32_t max2(uint32_t a, uint32_t b) {
    uint32_t d;
    asm("max.NaN.bf16x2 %0, %1, %2;" : "=r"(d) : "r"(a), "r"(b));
    return d;
  }
  __device__ static float amax(const uint4 v) {
    const uint32_t m = 0x7FFF7FFFu, w = max2(max2(v.x & m, v.y & m), max2(v.z & m, v.w & m));
    return max_nan(__uint_as_float(w << 16), __uint_as_float(w & 0xFFFF0000u));
  }
};
template <>
struct Vec<FI_DTYPE_F16> {
  static constexpr int kN = 8;
  __device__ static void unpack(const uint4 v, float* x) {
    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (int q = 0; q < 4; ++q) {
      x[2 * q] = f16_lo_to_f32(w[q]);
      x[2 * q + 1] = f16_hi_to_f32(w[q]);
    }
  }
  __device__ static uint32_t max2(uint32_t a, uint32_t b) {
    uint32_t d;
    asm("max.NaN.f16x2 %0, %1, %2;" : "=r"(d) : "r"(a), "r"(b));
    return d;
  }
  __device__ static float amax(const uint4 v) {
    const uint32_t m = 0x7FFF7FFFu, w = max2(max2(v.x & m, v.y & m), max2(v.z & m, v.w & m));
    return max_nan(f16_lo_to_f32(w), f16_hi_to_f32(w));
  }
};

// A block's scale and what its divisions need. Where the scale is far from the ends of the fp32
// range, x / scale is found as Markstein's theorem allows ("Computation of elementary functions on
// the IBM RISC System/6000 processor", 1990): with y the correctly rounded reciprocal and q within
// one unit of the quotient, q + (x - q scale) y rounds to the correctly rounded quotient. The
// first product may be two units off, so it takes two such steps: five packed instructions for
// two elements, where two IEEE divisions are several times that. All signs are turned, so that
// -0 keeps its own.
struct Scale {
  float s;
  uint64_t ss, my;  // (s, s), (-1 / s, -1 / s)
  bool plain;       // IEEE divisions
};

__device__ __forceinline__ Scale block_scale(float amax) {
  Scale r;
  r.s = __fdiv_rn(amax, 448.0f);
  r.plain = !(r.s > 0x1p-90f && r.s < 0x1p90f);
  const float y = -__frcp_rn(r.s);
  r.ss = pack2(r.s, r.s);
  r.my = pack2(y, y);
  return r;
}

__device__ __forceinline__ uint32_t quotient_codes(float x0, float x1, const Scale& s) {
  const uint64_t x = pack2(x0, x1);
  uint64_t q = mul2(x, s.my);
  q = fma2(fma2(q, s.ss, x), s.my, q);
  q = fma2(fma2(q, s.ss, x), s.my, q);
  float lo, hi;
  unpack2(q, lo, hi);
  return f32x2_to_e4m3x2(lo, hi);  // of the negative quotients
}

// kN codes of one 16-byte vector, stored at dst.
template <int DT>
__device__ __forceinline__ void store_codes(const uint4 v, const Scale& s, uint8_t* dst) {
  constexpr int kN = Vec<DT>::kN;
  float x[kN];
  Vec<DT>::unpack(v, x);
  uint32_t w[kN / 4];
  if (!s.plain) {
#pragma unroll
    for (int i = 0; i < kN / 4; ++i)
      w[i] = (quotient_codes(x[4 * i], x[4 * i + 1], s) | (quotient_codes(x[4 * i + 2], x[4 * i + 3], s) << 16)) ^
             0x80808080u;
  } else {
#pragma unroll
    for (int i = 0; i < kN / 4; ++i) {
      w[i] = 0;
      if (s.s != 0.0f)
        w[i] = f32x2_to_e4m3x2(__fdiv_rn(x[4 * i], s.s), __fdiv_rn(x[4 * i + 1], s.s)) |
               (f32x2_to_e4m3x2(__fdiv_rn(x[4 * i + 2], s.s), __fdiv_rn(x[4 * i + 3], s.s)) << 16);
    }
  }
  if constexpr (kN == 8)
    *reinterpret_cast<uint2*>(dst) = make_uint2(w[0], w[1]);
  else
    *reinterpret_cast<uint32_t*>(dst) = w[0];
}

// One group per 128 / kN lanes (16 lanes for 16-bit elements, a warp for fp32), U groups per
// lane so that U loads are in flight. WHOLE: k is a multiple of 128, so that the groups follow one
// another in memory and no row has to be found.
template <int DT, int U, bool WHOLE>
__global__ void __launch_bounds__(256, DT == FI_DTYPE_F32 ? 4 : 6)
    fp8_quant_rows_kernel(const uint8_t* __restrict__ x, int64_t groups, uint32_t kblocks, int64_t k,
                          uint8_t* __restrict__ q, float* __restrict__ scale) {
  constexpr int kN = Vec<DT>::kN, kLanes = kFp8Block / kN, kEs = 16 / kN;
  pdl_launch_dependents();
  pdl_wait();
  const int lane = threadIdx.x % kLanes;
  constexpr int kPerCta = 256 / kLanes;
  const int64_t g0 = (int64_t)blockIdx.x * kPerCta * U + threadIdx.x / kLanes;
  uint4 v[U];
  int64_t at[U];  // this lane's first element of the group; -1 behind the row's end
#pragma unroll
  for (int u = 0; u < U; ++u) {
    const int64_t g = g0 + u * kPerCta;
    if (WHOLE) {
      at[u] = g < groups ? g * kFp8Block + lane * kN : -1;
    } else {
      const int64_t row = groups <= 0x7fffffff ? (uint32_t)g / kblocks : g / kblocks;
      const int64_t e = (g - row * kblocks) * kFp8Block + lane * kN;
      at[u] = g < groups && e < k ? row * k + e : -1;
    }
    v[u] = make_uint4(0, 0, 0, 0);
    if (at[u] >= 0) v[u] = ldg_stream_v4(x + at[u] * kEs);
  }
#pragma unroll
  for (int u = 0; u < U; ++u) {
    float m = Vec<DT>::amax(v[u]);
#pragma unroll
    for (int o = kLanes / 2; o > 0; o >>= 1) m = max_nan(m, __shfl_xor_sync(0xffffffffu, m, o));
    const Scale s = block_scale(m);
    if (at[u] >= 0) store_codes<DT>(v[u], s, q + at[u]);
    if (lane == 0 && g0 + u * kPerCta < groups) scale[g0 + u * kPerCta] = s.s;
  }
}

// One CTA of 512 threads per 128 x 128 block, 32 elements per thread.
template <int DT>
__global__ void __launch_bounds__(512, DT == FI_DTYPE_F32 ? 2 : 4)
    fp8_quant_square_kernel(const uint8_t* __restrict__ x, int64_t rows, uint32_t kblocks, int64_t k,
                            uint8_t* __restrict__ q, float* __restrict__ scale) {
  constexpr int kN = Vec<DT>::kN, kLanes = kFp8Block / kN, kEs = 16 / kN, kU = 32 / kN;
  pdl_launch_dependents();
  pdl_wait();
  const int64_t rb = blockIdx.x / kblocks, cb = blockIdx.x - rb * kblocks;
  const int64_t e = cb * kFp8Block + (threadIdx.x % kLanes) * kN;
  const int64_t r0 = rb * kFp8Block + threadIdx.x / kLanes;
  constexpr int kStep = 512 / kLanes;  // rows per pass
  uint4 v[kU];
  float m = 0.0f;
#pragma unroll
  for (int u = 0; u < kU; ++u) {
    const int64_t r = r0 + u * kStep;
    v[u] = make_uint4(0, 0, 0, 0);
    if (r < rows && e < k) v[u] = ldg_stream_v4(x + (r * k + e) * kEs);
  }
#pragma unroll
  for (int u = 0; u < kU; ++u) m = max_nan(m, Vec<DT>::amax(v[u]));
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) m = max_nan(m, __shfl_xor_sync(0xffffffffu, m, o));
  __shared__ float warp_max[16];
  if ((threadIdx.x & 31) == 0) warp_max[threadIdx.x >> 5] = m;
  __syncthreads();
  m = warp_max[threadIdx.x & 15];
#pragma unroll
  for (int o = 8; o > 0; o >>= 1) m = max_nan(m, __shfl_xor_sync(0xffffffffu, m, o));
  const Scale s = block_scale(m);
#pragma unroll
  for (int u = 0; u < kU; ++u) {
    const int64_t r = r0 + u * kStep;
    if (r < rows && e < k) store_codes<DT>(v[u], s, q + r * k + e);
  }
  if (threadIdx.x == 0) scale[blockIdx.x] = s.s;
}

template <int DT>
int launch_quantize(const uint8_t* x, int64_t rows, int64_t k, bool square, uint8_t* q, float* scale,
                    cudaStream_t stream) {
  const int64_t kb = fp8_blocks(k);
  cudaLaunchConfig_t cfg = {};
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  if (square) {
    const int64_t grid = fp8_blocks(rows) * kb;
    if (grid > 0x7fffffffLL) return set_error(FI_ERR_UNSUPPORTED_SHAPE, "weight tensor too large");
    cfg.gridDim = dim3((unsigned)grid);
    cfg.blockDim = dim3(512);
    if (cudaLaunchKernelEx(&cfg, fp8_quant_square_kernel<DT>, x, rows, (uint32_t)kb, k, q, scale) != cudaSuccess)
      return set_cuda_error("fp8_quant_square_kernel launch");
    return FI_OK;
  }
  const int64_t groups = rows * kb, per_cta = 256 / (kFp8Block / Vec<DT>::kN);
  // four groups per lane once that still fills every SM with two CTAs, else one
  const bool deep = groups >= (int64_t)device_sm_count() * 2 * per_cta * 4;
  const int64_t grid = (groups + per_cta * (deep ? 4 : 1) - 1) / (per_cta * (deep ? 4 : 1));
  if (grid > 0x7fffffffLL) return set_error(FI_ERR_UNSUPPORTED_SHAPE, "activation tensor too large");
  cfg.gridDim = dim3((unsigned)grid);
  cfg.blockDim = dim3(256);
  const bool whole = k % kFp8Block == 0;
  auto kern = deep ? (whole ? fp8_quant_rows_kernel<DT, 4, true> : fp8_quant_rows_kernel<DT, 4, false>)
                   : (whole ? fp8_quant_rows_kernel<DT, 1, true> : fp8_quant_rows_kernel<DT, 1, false>);
  if (cudaLaunchKernelEx(&cfg, kern, x, groups, (uint32_t)kb, k, q, scale) != cudaSuccess)
    return set_cuda_error("fp8_quant_rows_kernel launch");
  return FI_OK;
}

}  // namespace

int launch_fp8_quantize(const void* x, int dtype, int64_t rows, int64_t k, bool square, uint8_t* q, float* scale,
                        cudaStream_t stream) {
  const uint8_t* p = static_cast<const uint8_t*>(x);
  switch (dtype) {
    case FI_DTYPE_BF16:
      return launch_quantize<FI_DTYPE_BF16>(p, rows, k, square, q, scale, stream);
    case FI_DTYPE_F16:
      return launch_quantize<FI_DTYPE_F16>(p, rows, k, square, q, scale, stream);
    default:
      return launch_quantize<FI_DTYPE_F32>(p, rows, k, square, q, scale, stream);
  }
}

}  // namespace fi
