// Device helpers and host-side tensor maps shared by the 8-bit product kernels.
#pragma once

#include <cstdint>
#include <cuda.h>

#include "common.cuh"
#include "internal.h"
#include "tc.cuh"

namespace fi {

// One test of the phase, suspended for as long as the hardware sees fit (microseconds, if the phase
// does not complete: nothing to look ahead with).
__device__ __forceinline__ bool mbar_test(uint32_t bar, uint32_t parity) {
  uint32_t done;
  asm volatile(
      "{\n .reg .pred p;\n mbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2;\n selp.u32 %0, 1, 0, p;\n}"
      : "=r"(done)
      : "r"(bar), "r"(parity)
      : "memory");
  return done != 0;
}

// mbar_wait_bounded (sync.cuh) for waits of a few hundred cycles: no time to suspend is named, so a
// waiting thread is back as soon as the hardware notices the phase, and the clock is read only in
// waits that have taken long. Once the CTA has aborted, the first test that fails is the last.
__device__ __forceinline__ bool mbar_wait_addr(uint32_t b, uint32_t parity, volatile int* abort_flag,
                                               uint64_t timeout_ns, unsigned* err_word, unsigned err_bit) {
  uint64_t t0 = 0;
#pragma unroll 1
  for (uint32_t i = 1;; ++i) {
    if (mbar_test(b, parity)) return true;
    if (i % 16 == 1 && *abort_flag) return false;
    if (i % 256 == 0) {  // reading the clock takes long: not in a wait that is about to end
      const uint64_t t = globaltimer_ns();
      if (t0 == 0) t0 = t;
      if (t - t0 > timeout_ns) {
        *abort_flag = 1;
        atomicOr(err_word, err_bit);
        return false;
      }
    }
  }
}

__device__ __forceinline__ bool mbar_wait_spin(uint64_t* bar, uint32_t parity, volatile int* abort_flag,
                                               uint64_t timeout_ns, unsigned* err_word, unsigned err_bit) {
  return mbar_wait_addr(smem_addr(bar), parity, abort_flag, timeout_ns, err_word, err_bit);
}

__device__ __forceinline__ void umma_f8(uint32_t d_tmem, uint64_t adesc, uint64_t bdesc, uint32_t idesc,
                                        uint32_t accumulate) {
  asm volatile(
      "{\n .reg .pred p;\n setp.ne.b32 p, %4, 0;\n tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], %1, %2, %3, p;\n}" ::"r"(
          d_tmem),
      "l"(adesc), "l"(bdesc), "r"(idesc), "r"(accumulate)
      : "memory");
}

// Instruction descriptor of kind::f8f6f4: fp32 accumulator (bits 4-5 = 1), E4M3 A and B (bits
// 7-9, 10-12 = 0), both K-major, N >> 3 in bits 17-22, M >> 4 in bits 24-28.
__device__ __forceinline__ constexpr uint32_t f8_idesc(int M, int N) {
  return (1u << 4) | ((uint32_t)(N >> 3) << 17) | ((uint32_t)(M >> 4) << 24);
}

__device__ __forceinline__ void tmem_ld_async(uint32_t taddr, uint32_t (&r)[16]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15}, "
      "[%16];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]),
        "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
      : "r"(taddr));
}

// Waits for this thread's TMEM loads; the registers they fill pass through it, so that no use of
// them can move above it.
__device__ __forceinline__ void tmem_wait_ld(uint32_t (&r)[16]) {
  asm volatile("tcgen05.wait::ld.sync.aligned;"
               : "+r"(r[0]), "+r"(r[1]), "+r"(r[2]), "+r"(r[3]), "+r"(r[4]), "+r"(r[5]), "+r"(r[6]), "+r"(r[7]),
                 "+r"(r[8]), "+r"(r[9]), "+r"(r[10]), "+r"(r[11]), "+r"(r[12]), "+r"(r[13]), "+r"(r[14]), "+r"(r[15])
               :
               : "memory");
}

__device__ __forceinline__ void tmem_ld_async(uint32_t taddr, uint32_t (&r)[32]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x32.b32 {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, "
      "%16, %17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31}, [%32];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]),
        "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15]), "=r"(r[16]),
        "=r"(r[17]), "=r"(r[18]), "=r"(r[19]), "=r"(r[20]), "=r"(r[21]), "=r"(r[22]), "=r"(r[23]), "=r"(r[24]),
        "=r"(r[25]), "=r"(r[26]), "=r"(r[27]), "=r"(r[28]), "=r"(r[29]), "=r"(r[30]), "=r"(r[31])
      : "r"(taddr));
}

__device__ __forceinline__ void tmem_wait_ld(uint32_t (&r)[32]) {
  asm volatile("tcgen05.wait::ld.sync.aligned;"
               : "+r"(r[0]), "+r"(r[1]), "+r"(r[2]), "+r"(r[3]), "+r"(r[4]), "+r"(r[5]), "+r"(r[6]), "+r"(r[7]),
                 "+r"(r[8]), "+r"(r[9]), "+r"(r[10]), "+r"(r[11]), "+r"(r[12]), "+r"(r[13]), "+r"(r[14]), "+r"(r[15]),
                 "+r"(r[16]), "+r"(r[17]), "+r"(r[18]), "+r"(r[19]), "+r"(r[20]), "+r"(r[21]), "+r"(r[22]),
                 "+r"(r[23]), "+r"(r[24]), "+r"(r[25]), "+r"(r[26]), "+r"(r[27]), "+r"(r[28]), "+r"(r[29]),
                 "+r"(r[30]), "+r"(r[31])
               :
               : "memory");
}

__device__ __forceinline__ void tmem_ld_async(uint32_t taddr, uint32_t (&r)[64]) {
  tmem_ld_async(taddr, *reinterpret_cast<uint32_t(*)[32]>(r));
  tmem_ld_async(taddr + 32, *reinterpret_cast<uint32_t(*)[32]>(r + 32));
}

__device__ __forceinline__ void tmem_wait_ld(uint32_t (&r)[64]) {
  tmem_wait_ld(*reinterpret_cast<uint32_t(*)[32]>(r));
  tmem_wait_ld(*reinterpret_cast<uint32_t(*)[32]>(r + 32));  // at once: nothing is under way any more
}

// (x, y) += (a, b) * (s.x, s.y), both lanes of one packed instruction.
__device__ __forceinline__ void fma_scaled(float& x, float& y, uint32_t a, uint32_t b, uint64_t s) {
  asm("{\n .reg .b64 d, f;\n mov.b64 d, {%2, %3};\n mov.b64 f, {%0, %1};\n fma.rn.f32x2 f, d, %4, f;\n"
      " mov.b64 {%0, %1}, f;\n}"
      : "+f"(x), "+f"(y)
      : "r"(a), "r"(b), "l"(s));
}

// Four fp32 at `addr` (a shared-memory address of this CTA) in the cluster's CTA `rank`.
__device__ __forceinline__ float4 ld_dsmem_v4(uint32_t addr, uint32_t rank) {
  uint32_t remote;
  float4 v;
  asm("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(remote) : "r"(addr), "r"(rank));
  asm volatile("ld.shared::cluster.v4.f32 {%0, %1, %2, %3}, [%4];"
               : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w)
               : "r"(remote));
  return v;
}

__device__ __forceinline__ void store_out(void* out, int dtype, int64_t at, float v) {
  if (dtype == FI_DTYPE_F32)
    static_cast<float*>(out)[at] = v;
  else
    static_cast<uint16_t*>(out)[at] = f32_to_out(v, dtype == FI_DTYPE_F16);
}

// Up to four consecutive outputs (`left` of them inside the row); wide: aligned, one store.
__device__ __forceinline__ void store_out4(void* out, int dtype, int64_t at, float4 v, bool wide, int64_t left) {
  if (wide && left >= 4) {
    if (dtype == FI_DTYPE_F32)
      *reinterpret_cast<float4*>(static_cast<float*>(out) + at) = v;
    else
      *reinterpret_cast<uint2*>(static_cast<uint16_t*>(out) + at) =
          dtype == FI_DTYPE_F16 ? make_uint2(f32x2_to_f16x2(v.x, v.y), f32x2_to_f16x2(v.z, v.w))
                                : make_uint2(f32x2_to_bf16x2(v.x, v.y), f32x2_to_bf16x2(v.z, v.w));
    return;
  }
  store_out(out, dtype, at, v.x);
  if (left > 1) store_out(out, dtype, at + 1, v.y);
  if (left > 2) store_out(out, dtype, at + 2, v.z);
  if (left > 3) store_out(out, dtype, at + 3, v.w);
}

// (a, b) = (silu(a) u, silu(b) v) with silu(g) = g / (1 + exp(-g)) through e = exp(-|g|), which cannot overflow:
// g e / (1 + e) where g < 0. The activation is off by at most 7 units (2^-23) of itself for every g, and by
// a few of 2^-149 where it is subnormal. e is 2^t corrected by what t = -|g| log2 e lost in its rounding, as it is
// up to 150; 2^64 e below t = -64, since the instruction gives 0 for what is subnormal. (With expf and an IEEE
// division, 64 times a thread in the CTA-pair kernel, whose instructions come from far, 8192 x 20000 x 128 gated
// took 500 us.)
__device__ __forceinline__ void silu_times(float& a, float& b, float u, float v) {
  constexpr float kLog2e = 1.4426950408889634f, kLn2 = 0.6931471805599453f;
  constexpr float kLn2Rest = (float)(0.6931471805599453 - (double)kLn2);
  const uint64_t x = pack2(fmaxf(-fabsf(a), -200.0f), fmaxf(-fabsf(b), -200.0f));
  const uint64_t t = mul2(x, pack2(kLog2e, kLog2e));
  const uint64_t lost = fma2(t, pack2(-kLn2Rest, -kLn2Rest), fma2(t, pack2(-kLn2, -kLn2), x));
  float t0, t1, e0, e1, d0, d1, r0, r1;
  unpack2(t, t0, t1);
  const bool far0 = t0 < -64.0f, far1 = t1 < -64.0f;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(e0) : "f"(far0 ? t0 + 64.0f : t0));
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(e1) : "f"(far1 ? t1 + 64.0f : t1));
  const uint64_t e2 = pack2(e0, e1), e = fma2(e2, lost, e2);
  const uint64_t back = pack2(far0 ? 0x1p-64f : 1.0f, far1 ? 0x1p-64f : 1.0f);
  unpack2(fma2(e, back, pack2(1.0f, 1.0f)), d0, d1);
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r0) : "f"(d0));
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r1) : "f"(d1));
  unpack2(mul2(mul2(pack2(a, b), e), back), d0, d1);
  unpack2(mul2(mul2(pack2(a < 0.0f ? d0 : a, b < 0.0f ? d1 : b), pack2(r0, r1)), pack2(u, v)), a, b);
}

// Codes [rows, k] in boxes of 128 k x box_rows, 128-byte swizzle; what is outside reads as zero.
inline int encode_codes(CUtensorMap* map, const uint8_t* base, int64_t k, int64_t rows, int box_rows) {
  const uint64_t dims[2] = {(uint64_t)k, (uint64_t)rows};
  const uint64_t strides[1] = {(uint64_t)k};
  const uint32_t box[2] = {(uint32_t)kFp8Block, (uint32_t)box_rows};
  return encode_tensor_map(map, CU_TENSOR_MAP_DATA_TYPE_UINT8, 2, base, dims, strides, box,
                           CU_TENSOR_MAP_SWIZZLE_128B);
}

}  // namespace fi
