// Log probabilities of given tokens, with entropy, rank and the greatest alternatives.
//
// Per row z of logits, in one pass over it:
//   M = max z, S = sum exp(z - M), T = sum (z - M) exp(z - M)
//   logprob = (z[t] - M) - ln S,  entropy = ln S - T / S,
//   rank = entries before t in the order (value descending, NaN first; index ascending),
//   top  = the first K of that order.
//
// Each thread keeps a running (M, S, T) and rescales when its maximum grows: with the new
// maximum M', c = exp(M - M'), S' = c S and T' = c (T + (M - M') S). Each warp keeps the best 32
// keys it has seen, one per lane in order; an element above the K-th of them goes to the warp's
// buffer in shared memory, and 32 buffered keys at a time are sorted (bitonic, by shuffles) and
// merged into the list. A key is the value as an order-preserving 32-bit integer above the
// inverted index, so equal values order by index and every result is the same from run to run.
//
// A row is one CTA, or one cluster of CTAs when there are few rows; the CTAs' sums and lists
// meet in distributed shared memory. No workspace, no atomics on global memory.
//
// Masked entries: -inf is replaced by a value so low that its exponential is 0 (kFloor), which
// keeps (z - M) exp(z - M) at 0 instead of NaN. A row whose maximum is not above that value (all
// entries masked, or masks of the type's lowest value only) or is beyond +1e38 is summed
// again with every difference clamped.
#include <cstdint>
#include <algorithm>

#include "common.cuh"
#include "internal.h"
#include "sync.cuh"

namespace fi {

namespace {

constexpr int kThreads = 256, kWarps = kThreads / 32;
constexpr int kBuffer = 32 + 256;  // keys a warp may hold before it merges: 31, and one vector of every lane
constexpr float kLog2e = 1.4426950408889634f, kLn2 = 0.6931471805599453f;
constexpr float kFloor = -1e38f;  // stands for -inf: (kFloor - M) log2 e is finite, its exponential 0
constexpr float kFar = -1e30f;    // least difference of two maxima: times a sum it stays finite

__device__ __forceinline__ float max_nan(float a, float b) {
  float d;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(d) : "f"(a), "f"(b));
  return d;
}

__device__ __forceinline__ float exp2_fast(float x) {
  float d;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(d) : "f"(x));
  return d;
}

// Order-preserving integer of a logit: NaN above everything, -0 equal to +0.
__device__ __forceinline__ uint32_t order_of(float x) {
  if (x != x) return 0xFFFFFFFFu;
  const uint32_t b = __float_as_uint(x + 0.0f);
  return b & 0x80000000u ? ~b : b | 0x80000000u;
}

__device__ __forceinline__ float value_of(uint32_t order) {
  if (order == 0xFFFFFFFFu) return __uint_as_float(0x7FC00000u);
  return __uint_as_float(order & 0x80000000u ? order & 0x7FFFFFFFu : ~order);
}

// Greater is earlier in the order. 0 is below every key.
__device__ __forceinline__ uint64_t key_of(float x, uint32_t index) {
  return (uint64_t)order_of(x) << 32 | (uint32_t)~index;
}

template <int DT>
struct Elem;
template <>
struct Elem<FI_DTYPE_F32> {
  using T = float;
  static constexpr int kN = 4;
  __device__ static float get(const uint32_t (&w)[4], int i) { return __uint_as_float(w[i]); }
  __device__ static float one(const void* p, int64_t i) { return static_cast<const float*>(p)[i]; }
};
template <>
struct Elem<FI_DTYPE_BF16> {
  using T = uint16_t;
  static constexpr int kN = 8;
  __device__ static float get(const uint32_t (&w)[4], int i) {
    return __uint_as_float(i & 1 ? w[i / 2] & 0xFFFF0000u : w[i / 2] << 16);
  }
  __device__ static float one(const void* p, int64_t i) { return bf16_bits_to_f32(static_cast<const uint16_t*>(p)[i]); }
};
template <>
struct Elem<FI_DTYPE_F16> {
  using T = uint16_t;
  static constexpr int kN = 8;
  __device__ static float get(const uint32_t (&w)[4], int i) {
    return i & 1 ? f16_hi_to_f32(w[i / 2]) : f16_lo_to_f32(w[i / 2]);
  }
  __device__ static float one(const void* p, int64_t i) { return f16_lo_to_f32(static_cast<const uint16_t*>(p)[i]); }
};

struct Sums {
  float m, s, t;  // maximum, sum of 2^((z - m) log2 e), sum of (z - m) times that
};

__device__ __forceinline__ Sums join(const Sums a, const Sums b) {
  Sums r;
  r.m = max_nan(a.m, b.m);
  const float da = max_nan(a.m - r.m, kFar), db = max_nan(b.m - r.m, kFar);
  const float ca = exp2_fast(da * kLog2e), cb = exp2_fast(db * kLog2e);
  r.s = ca * a.s + cb * b.s;
  r.t = ca * (a.t + da * a.s) + cb * (b.t + db * b.s);
  return r;
}

__device__ __forceinline__ uint64_t shfl_xor64(uint64_t v, int o) { return __shfl_xor_sync(0xffffffffu, v, o); }

// The warp's 32 keys, one per lane, into ascending order by lane.
__device__ __forceinline__ uint64_t sort32(uint64_t v, int lane) {
#pragma unroll
  for (int size = 2; size <= 32; size *= 2)
#pragma unroll
    for (int o = size / 2; o > 0; o /= 2) {
      const uint64_t w = shfl_xor64(v, o);
      const bool up = (lane & size) == 0 || size == 32;
      const bool low = (lane & o) == 0;
      v = (low == up) == (v < w) ? v : w;
    }
  return v;
}

// The 32 greatest of a descending list and an ascending one, descending.
__device__ __forceinline__ uint64_t merge32(uint64_t list, uint64_t asc, int lane) {
  uint64_t v = list > asc ? list : asc;
#pragma unroll
  for (int o = 16; o > 0; o /= 2) {
    const uint64_t w = shfl_xor64(v, o);
    v = ((lane & o) == 0) == (v > w) ? v : w;
  }
  return v;
}

__device__ __forceinline__ void cluster_sync() {
  asm volatile("barrier.cluster.arrive.release.aligned;\nbarrier.cluster.wait.acquire.aligned;" ::: "memory");
}

__device__ __forceinline__ uint32_t ld_dsmem_u32(const void* p, uint32_t rank) {
  uint32_t remote, v;
  asm("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(remote) : "r"(smem_addr(p)), "r"(rank));
  asm volatile("ld.shared::cluster.u32 %0, [%1];" : "=r"(v) : "r"(remote));
  return v;
}

__device__ __forceinline__ uint64_t ld_dsmem_u64(const void* p, uint32_t rank) {
  uint32_t remote;
  uint64_t v;
  asm("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(remote) : "r"(smem_addr(p)), "r"(rank));
  asm volatile("ld.shared::cluster.u64 %0, [%1];" : "=l"(v) : "r"(remote));
  return v;
}

template <int DT>
__global__ void __launch_bounds__(kThreads) token_logprobs_kernel(const LogprobArgs p, int ctas) {
  using E = Elem<DT>;
  constexpr int kN = E::kN;
  __shared__ uint64_t buffers[kWarps][kBuffer];
  __shared__ uint32_t counts[kWarps];
  __shared__ uint64_t lists[kWarps][32];
  __shared__ float sums[kWarps][3];
  __shared__ uint32_t before[kWarps];
  __shared__ struct {
    uint64_t list[32];
    float m, s, t;
    uint32_t before;
  } cta;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int part = (int)(blockIdx.x % (unsigned)ctas);
  const int64_t row = blockIdx.x / (unsigned)ctas;
  const int K = p.topk;
  pdl_launch_dependents();
  if (lane == 0) counts[warp] = 0;
  __syncwarp();
  pdl_wait();
  const typename E::T* z = static_cast<const typename E::T*>(p.logits) + row * p.ld;
  const int vocab = (int)p.vocab;
  const int64_t token = p.tokens[row];
  const bool has_token = token >= 0 && token < p.vocab;
  const float zt = has_token ? E::one(z, token) : 0.0f;
  const uint64_t token_key = has_token ? key_of(zt, (uint32_t)token) : 0;

  // vector v covers elements [v kN - shift, + kN): 16-byte aligned in memory
  const int shift = (int)((reinterpret_cast<uintptr_t>(z) & 15) / sizeof(typename E::T));
  const int64_t vectors = ((int64_t)vocab + shift + kN - 1) / kN;

  Sums a{kFloor, 0.0f, 0.0f};
  uint32_t earlier = 0;                      // entries before the token
  uint64_t list = 0;                         // this lane's entry of the warp's best, descending by lane
  uint64_t least = 0;                        // the K-th of them
  float above = K > 0 ? __uint_as_float(0x7FC00000u) : __uint_as_float(0x7F800000u);  // its value; NaN: none yet

  auto flush = [&](uint32_t count) {  // merge `count` buffered keys into the list
    for (uint32_t i = 0; i < count; i += 32) {
      const uint64_t v = i + lane < count ? buffers[warp][i + lane] : 0;
      list = merge32(list, sort32(v, lane), lane);
    }
    least = __shfl_sync(0xffffffffu, list, K - 1);
    if (least != 0) above = value_of((uint32_t)(least >> 32));
    __syncwarp();
    if (lane == 0) counts[warp] = 0;
    __syncwarp();
  };

  const int64_t step = (int64_t)ctas * kThreads;
  const int64_t warp0 = (int64_t)part * kThreads + warp * 32;
  for (int64_t v0 = warp0; v0 < vectors; v0 += step) {
    const int64_t v = v0 + lane;
    const int e0 = (int)(v * kN) - shift;
    uint32_t w[4] = {0, 0, 0, 0};
    const bool whole = v < vectors && e0 >= 0 && e0 + kN <= vocab;
    if (whole) {
      const uint4 q = ldg_stream_v4(z + e0);
      w[0] = q.x;
      w[1] = q.y;
      w[2] = q.z;
      w[3] = q.w;
    }
    float x[kN];
#pragma unroll
    for (int i = 0; i < kN; ++i) x[i] = E::get(w, i);
    uint32_t valid = (1u << kN) - 1;
    if (!whole) {  // the row's ends, element by element; what is outside it counts as masked
      valid = 0;
#pragma unroll
      for (int i = 0; i < kN; ++i) {
        const bool in = v < vectors && e0 + i >= 0 && e0 + i < vocab;
        x[i] = in ? E::one(z, e0 + i) : __uint_as_float(0xFF800000u);
        valid |= in ? 1u << i : 0;
      }
    }
    float mx = x[0];
#pragma unroll
    for (int i = 1; i < kN; ++i) mx = max_nan(mx, x[i]);
    if (mx > a.m) {
      const float d = max_nan(a.m - mx, kFar);
      const float c = exp2_fast(d * kLog2e);
      a.t = c * (a.t + d * a.s);
      a.s = c * a.s;
      a.m = mx;
    }
#pragma unroll
    for (int i = 0; i < kN; ++i) {
      const float d = max_nan(x[i], kFloor) - a.m;
      const float e = exp2_fast(d * kLog2e);
      a.s += valid >> i & 1 ? e : 0.0f;
      a.t = fmaf(d, valid >> i & 1 ? e : 0.0f, a.t);
    }
    if (has_token && !(mx < zt)) {
#pragma unroll
      for (int i = 0; i < kN; ++i)
        earlier += (valid >> i & 1) && key_of(x[i], (uint32_t)(e0 + i)) > token_key ? 1 : 0;
    }
    // buffer what is above the warp's K-th (a NaN compares as above)
    const bool any = K > 0 && valid != 0 && !(mx <= above);
    if (__any_sync(0xffffffffu, any)) {
      if (any) {
#pragma unroll
        for (int i = 0; i < kN; ++i) {
          const uint64_t key = key_of(x[i], (uint32_t)(e0 + i));
          if ((valid >> i & 1) && key > least) buffers[warp][atomicAdd(&counts[warp], 1u)] = key;
        }
      }
      __syncwarp();
      const uint32_t count = counts[warp];
      if (count >= 32) flush(count);
    }
  }
  if (K > 0) {
    __syncwarp();
    flush(counts[warp]);
    lists[warp][lane] = list;
  }
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) {
    Sums b;
    b.m = __shfl_xor_sync(0xffffffffu, a.m, o);
    b.s = __shfl_xor_sync(0xffffffffu, a.s, o);
    b.t = __shfl_xor_sync(0xffffffffu, a.t, o);
    // the same order on both sides of the exchange, so that all lanes agree in every bit
    a = lane & o ? join(b, a) : join(a, b);
    earlier += __shfl_xor_sync(0xffffffffu, earlier, o);
  }
  if (lane == 0) {
    sums[warp][0] = a.m;
    sums[warp][1] = a.s;
    sums[warp][2] = a.t;
    before[warp] = earlier;
  }
  __syncthreads();
  if (warp == 0) {
    a = Sums{sums[0][0], sums[0][1], sums[0][2]};
    earlier = before[0];
    for (int w = 1; w < kWarps; ++w) {
      a = join(a, Sums{sums[w][0], sums[w][1], sums[w][2]});
      earlier += before[w];
      if (K > 0) list = merge32(list, lists[w][31 - lane], lane);
    }
    if (ctas > 1) {
      cta.list[lane] = list;
      if (lane == 0) {
        cta.m = a.m;
        cta.s = a.s;
        cta.t = a.t;
        cta.before = earlier;
      }
    }
  }
  if (ctas > 1) {
    __syncwarp();
    cluster_sync();
    if (part == 0 && warp == 0) {
      for (int r = 1; r < ctas; ++r) {
        a = join(a, Sums{__uint_as_float(ld_dsmem_u32(&cta.m, r)), __uint_as_float(ld_dsmem_u32(&cta.s, r)),
                         __uint_as_float(ld_dsmem_u32(&cta.t, r))});
        earlier += ld_dsmem_u32(&cta.before, r);
        if (K > 0) list = merge32(list, ld_dsmem_u64(&cta.list[31 - lane], r), lane);
      }
    }
    __syncwarp();
    cluster_sync();  // no CTA leaves while its sums are read
    if (part != 0) return;
  }
  __syncthreads();
  if (threadIdx.x == 0) {
    cta.m = a.m;
    cta.s = a.s;
    cta.t = a.t;
  }
  __syncthreads();
  a = Sums{cta.m, cta.s, cta.t};
  if (a.m <= kFloor || a.m > 1e38f) {
    // rare: the true maximum first, then sums with clamped differences, by this CTA alone
    float mx = __uint_as_float(0xFF800000u);
    for (int i = threadIdx.x; i < vocab; i += kThreads) mx = max_nan(mx, E::one(z, i));
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) mx = max_nan(mx, __shfl_xor_sync(0xffffffffu, mx, o));
    if (lane == 0) sums[warp][0] = mx;
    __syncthreads();
    for (int w = 0; w < kWarps; ++w) mx = max_nan(mx, sums[w][0]);
    __syncthreads();
    float s = 0.0f, t = 0.0f;
    for (int i = threadIdx.x; i < vocab; i += kThreads) {
      const float x = E::one(z, i);
      if (x != __uint_as_float(0xFF800000u)) {
        const float d = max_nan(x - mx, kFar);
        const float e = exp2_fast(d * kLog2e);
        s += e;
        t = fmaf(d, e, t);
      }
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) {
      s += __shfl_xor_sync(0xffffffffu, s, o);
      t += __shfl_xor_sync(0xffffffffu, t, o);
    }
    if (lane == 0) {
      sums[warp][1] = s;
      sums[warp][2] = t;
    }
    __syncthreads();
    a = Sums{mx, 0.0f, 0.0f};
    for (int w = 0; w < kWarps; ++w) {
      a.s += sums[w][1];
      a.t += sums[w][2];
    }
  }
  if (warp != 0) return;
  const bool empty = a.s == 0.0f;  // nothing but -inf
  const float ln_s = empty ? 0.0f : __log2f(a.s) * kLn2;
  auto logprob_of = [&](float x) { return empty ? x : (x - a.m) - ln_s; };
  if (lane == 0) {
    p.logprob[row] = has_token ? logprob_of(zt) : __uint_as_float(0x7FC00000u);
    p.entropy[row] = empty ? 0.0f : ln_s - a.t / a.s;
    p.rank[row] = has_token ? (int64_t)earlier : -1;
  }
  if (lane < K) {
    p.top_logprobs[row * K + lane] = logprob_of(value_of((uint32_t)(list >> 32)));
    p.top_ids[row * K + lane] = (int64_t)(uint32_t)~(uint32_t)list;
  }
}

template <int DT>
int launch(const LogprobArgs& a, cudaStream_t stream) {
  // CTAs per row: as many as leave each at least 4 vectors per thread, while the rows alone do
  // not give every SM its CTAs
  const int64_t vectors = a.vocab / Elem<DT>::kN;
  int ctas = 1;
  while (ctas < 8 && a.rows * ctas * 2 <= (int64_t)device_sm_count() * 4 && vectors >= (int64_t)ctas * 2 * kThreads * 4)
    ctas *= 2;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = (unsigned)ctas;
  attr[1].val.clusterDim.y = 1;
  attr[1].val.clusterDim.z = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)(a.rows * ctas));
  cfg.blockDim = dim3(kThreads);
  cfg.stream = stream;
  cfg.attrs = attr;
  cfg.numAttrs = 2;
  if (cudaLaunchKernelEx(&cfg, token_logprobs_kernel<DT>, a, ctas) != cudaSuccess)
    return set_cuda_error("token_logprobs_kernel launch");
  return FI_OK;
}

}  // namespace

int launch_token_logprobs(const LogprobArgs& a, int dtype, cudaStream_t stream) {
  switch (dtype) {
    case FI_DTYPE_BF16:
      return launch<FI_DTYPE_BF16>(a, stream);
    case FI_DTYPE_F16:
      return launch<FI_DTYPE_F16>(a, stream);
    default:
      return launch<FI_DTYPE_F32>(a, stream);
  }
}

}  // namespace fi
