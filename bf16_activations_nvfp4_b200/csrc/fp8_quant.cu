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
// codes. HBM-bound: element bytes + 1 per element.
#include <cstdint>

#include "common.cuh"
#include "internal.h"

namespace fi {

namespace {

__device__ __forceinline__ float max_nan(float a, float b) {
  float d;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(d) : "f"(a), "f"(b));
  return d;
}

// Two fp32 values to two E4M3 codes (low byte = lo), round to nearest even, saturating.
__device__ __forceinline__ uint32_t f32x2_to_e4m3x2(float lo, float hi) {
  unsigned short r;
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(r) : "f"(hi), "f"(lo));
  return r;
}

// 16 bytes of input as fp32 (DT = fi_dtype).
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
};

__device__ __forceinline__ float block_scale(float amax) { return __fdiv_rn(amax, 448.0f); }

// kN codes of one 16-byte vector, stored at dst.
template <int DT>
__device__ __forceinline__ void store_codes(const uint4 v, float scale, uint8_t* dst) {
  constexpr int kN = Vec<DT>::kN;
  float x[kN];
  Vec<DT>::unpack(v, x);
  uint32_t w[kN / 4];
#pragma unroll
  for (int i = 0; i < kN / 4; ++i) {
    w[i] = 0;
    if (scale != 0.0f)
      w[i] = f32x2_to_e4m3x2(__fdiv_rn(x[4 * i], scale), __fdiv_rn(x[4 * i + 1], scale)) |
             (f32x2_to_e4m3x2(__fdiv_rn(x[4 * i + 2], scale), __fdiv_rn(x[4 * i + 3], scale)) << 16);
  }
  if constexpr (kN == 8)
    *reinterpret_cast<uint2*>(dst) = make_uint2(w[0], w[1]);
  else
    *reinterpret_cast<uint32_t*>(dst) = w[0];
}

template <int DT>
__device__ __forceinline__ float vec_amax(const uint4 v) {
  float x[Vec<DT>::kN];
  Vec<DT>::unpack(v, x);
  float m = 0.0f;
#pragma unroll
  for (int i = 0; i < Vec<DT>::kN; ++i) m = max_nan(m, fabsf(x[i]));
  return m;
}

// One group per 128 / kN lanes (16 lanes for 16-bit elements, a warp for fp32), U groups per
// lane so that U loads are in flight.
template <int DT, int U>
__global__ void __launch_bounds__(256) fp8_quant_rows_kernel(const uint8_t* __restrict__ x, int64_t groups,
                                                             uint32_t kblocks, int64_t k, uint8_t* __restrict__ q,
                                                             float* __restrict__ scale) {
  constexpr int kN = Vec<DT>::kN, kLanes = kFp8Block / kN, kEs = 16 / kN;
  pdl_launch_dependents();
  pdl_wait();
  const int lane = threadIdx.x % kLanes;
  const int64_t per_cta = 256 / kLanes;
  const int64_t g0 = (int64_t)blockIdx.x * per_cta * U + threadIdx.x / kLanes;
  uint4 v[U];
#pragma unroll
  for (int u = 0; u < U; ++u) {
    const int64_t g = g0 + u * per_cta;
    const int64_t row = g / kblocks, e = (g - row * kblocks) * kFp8Block + lane * kN;
    v[u] = make_uint4(0, 0, 0, 0);
    if (g < groups && e < k) v[u] = ldg_stream_v4(x + (row * k + e) * kEs);
  }
#pragma unroll
  for (int u = 0; u < U; ++u) {
    const int64_t g = g0 + u * per_cta;
    const int64_t row = g / kblocks, e = (g - row * kblocks) * kFp8Block + lane * kN;
    float m = vec_amax<DT>(v[u]);
#pragma unroll
    for (int o = kLanes / 2; o > 0; o >>= 1) m = max_nan(m, __shfl_xor_sync(0xffffffffu, m, o));
    const float s = block_scale(m);
    if (g < groups) {
      if (e < k) store_codes<DT>(v[u], s, q + row * k + e);
      if (lane == 0) scale[g] = s;
    }
  }
}

// One CTA of 512 threads per 128 x 128 block, 32 elements per thread.
template <int DT>
__global__ void __launch_bounds__(512) fp8_quant_square_kernel(const uint8_t* __restrict__ x, int64_t rows,
                                                               uint32_t kblocks, int64_t k, uint8_t* __restrict__ q,
                                                               float* __restrict__ scale) {
  constexpr int kN = Vec<DT>::kN, kLanes = kFp8Block / kN, kEs = 16 / kN, kU = 32 / kN;
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
  for (int u = 0; u < kU; ++u) m = max_nan(m, vec_amax<DT>(v[u]));
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) m = max_nan(m, __shfl_xor_sync(0xffffffffu, m, o));
  __shared__ float warp_max[16];
  if ((threadIdx.x & 31) == 0) warp_max[threadIdx.x >> 5] = m;
  __syncthreads();
  m = warp_max[threadIdx.x & 15];
#pragma unroll
  for (int o = 8; o > 0; o >>= 1) m = max_nan(m, __shfl_xor_sync(0xffffffffu, m, o));
  const float s = block_scale(m);
#pragma unroll
  for (int u = 0; u < kU; ++u) {
    const int64_t r = r0 + u * kStep;
    if (r < rows && e < k) store_codes<DT>(v[u], s, q + r * k + e);
  }
  if (threadIdx.x == 0) scale[blockIdx.x] = s;
}

template <int DT>
int launch_quantize(const uint8_t* x, int64_t rows, int64_t k, bool square, uint8_t* q, float* scale,
                    cudaStream_t stream) {
  const int64_t kb = fp8_blocks(k);
  if (square) {
    const int64_t grid = fp8_blocks(rows) * kb;
    if (grid > 0x7fffffffLL) return set_error(FI_ERR_UNSUPPORTED_SHAPE, "weight tensor too large");
    fp8_quant_square_kernel<DT><<<(unsigned)grid, 512, 0, stream>>>(x, rows, (uint32_t)kb, k, q, scale);
    if (cudaGetLastError() != cudaSuccess) return set_cuda_error("fp8_quant_square_kernel launch");
    return FI_OK;
  }
  const int64_t groups = rows * kb, per_cta = 256 / (kFp8Block / Vec<DT>::kN);
  // four groups per lane once that still fills every SM with two CTAs, else one
  const bool deep = groups >= (int64_t)device_sm_count() * 2 * per_cta * 4;
  const int64_t grid = (groups + per_cta * (deep ? 4 : 1) - 1) / (per_cta * (deep ? 4 : 1));
  if (grid > 0x7fffffffLL) return set_error(FI_ERR_UNSUPPORTED_SHAPE, "activation tensor too large");
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)grid);
  cfg.blockDim = dim3(256);
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  if (cudaLaunchKernelEx(&cfg, deep ? fp8_quant_rows_kernel<DT, 4> : fp8_quant_rows_kernel<DT, 1>, x, groups,
                         (uint32_t)kb, k, q, scale) != cudaSuccess)
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
