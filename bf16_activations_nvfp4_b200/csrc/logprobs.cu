// Log probabilities of given tokens, with entropy, rank and the greatest alternatives.
//
// Per row z of logits, in one pass over it:
//   M = max z, S = sum exp(z - M), T = sum (z - M) exp(z - M)
//   logprob = (z[t] - M) - ln S,  entropy = ln S - T / S,
//   rank = entries before t in the order (value descending, NaN first; index ascending),
//   top  = the first K of that order.
//
// Each thread keeps a running (M, S, T) and rescales when its maximum grows: with the new
// maximum M', c = exp(M - M'), S' = c S and T' = c (T + (M - M') S). The rank counts greater elements
// by packed comparisons.
//
// Candidates for the list are keys: the value as an order-preserving 32-bit integer above the
// inverted index, so equal values order by index and every result is the same from run to run.
// Only an element above a limit becomes one: the K-th of the threads' (or of 32 groups of threads')
// maxima so far, found up to four times per row, as at least K elements are not below it and few
// more are. A warp's candidates go to its buffer in shared memory; 32 of them are sorted (bitonic,
// by shuffles) and merged into its list of the best 32, one per lane. Mostly there are fewer: then
// those of all warps are put in a row at the end and take one sort.
//
// A row is one CTA, or one cluster of CTAs when there are few rows; the CTAs' sums and lists
// meet in distributed shared memory. No workspace, no atomics.
//
// 2047 x 152064 bf16 takes 99 us without token or list (6.3 TB/s), 117 with ranks, 147 with 5
// alternatives, 212 with 32: bound by HBM, then by instruction issue (73% of the slots, at 24 warps
// per SM) and the latency of the lists' steps, during which a warp's next groups are on their way to
// shared memory (held in registers instead, one group ahead, and candidates inserted one by one it
// was 111, 131, 186 and 262). 1024 x 152064 fp32 with 5 takes 122 us, 4096 x 32000 bf16 with 5 89
// (inserted one by one: 117). One fp32 row of 152064 with 20 takes 13 us, most of it the latency of
// the steps at its end (6.1 without the list).
//
// Masked entries: -inf, and what is below -2^26, is replaced by that value (kFloor), whose exponential
// is 0 next to any maximum from -2^24 on; (z - M) exp(z - M) stays 0 instead of NaN. M log2 e is
// rounded, by up to 1 at 2^24: the exponentials are off by that power of two, which ln S takes back.
// A row whose maximum is of a greater magnitude (all entries masked, too) is summed again with exact
// and clamped differences.
#include <cstdint>
#include <algorithm>
#include <atomic>

#include "common.cuh"
#include "internal.h"
#include "sync.cuh"

namespace fi {

namespace {

constexpr int kBuffer = 64;  // keys a warp may hold before it merges: 31, and one of every lane
constexpr int kMaxCtas = 8;  // of a row: a portable cluster
constexpr int kSlots = 3;     // groups of vectors per warp that are on their way, or being used
constexpr int kU = 4;         // vectors of a lane in a group
constexpr int kFewTops = 8;   // up to here a limit comes from 32 maxima
constexpr int kShort = 128, kMany = 256, kFew = 1024;  // threads of a CTA: many rows, rows, few long rows
constexpr float kLog2e = 1.4426950408889634f, kLn2 = 0.6931471805599453f;
constexpr float kFloor = -0x1p26f;  // stands for -inf and all below it (0xCC80 in bf16)
constexpr float kFarMax = 0x1p24f;  // a greater magnitude of the row's maximum takes a second pass
constexpr float kFar = -1e30f;    // least difference of two maxima: times a sum it stays finite

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

// The value just below x (x finite or +inf); NaN for -inf, which has none, and for NaN.
__device__ __forceinline__ float below(float x) {
  const uint32_t b = __float_as_uint(x + 0.0f);
  if (!(x > __uint_as_float(0xFF800000u))) return __uint_as_float(0x7FC00000u);
  return __uint_as_float(b == 0 ? 0x80000001u : (b & 0x80000000u ? b + 1 : b - 1));
}

// The same of 16-bit floating-point bits, `lowest` those of -inf.
__device__ __forceinline__ uint32_t below16(uint32_t b, uint32_t lowest) {
  b = b == 0x8000u ? 0u : b;
  if (b == lowest || (b & 0x7FFFu) > (lowest & 0x7FFFu)) return 0x7FFFu;  // a NaN
  return b == 0 ? 0x8001u : (b & 0x8000u ? b + 1 : b - 1);
}

__device__ __forceinline__ uint32_t max_bf16x2(uint32_t a, uint32_t b) {
  uint32_t d;
  asm("max.NaN.bf16x2 %0, %1, %2;" : "=r"(d) : "r"(a), "r"(b));
  return d;
}

__device__ __forceinline__ uint32_t max_f16x2(uint32_t a, uint32_t b) {
  uint32_t d;
  asm("max.NaN.f16x2 %0, %1, %2;" : "=r"(d) : "r"(a), "r"(b));
  return d;
}

// w[i], i not known at compile time.
__device__ __forceinline__ uint32_t word_of(const uint32_t (&w)[4], int i) {
  const uint32_t lo = i & 1 ? w[1] : w[0], hi = i & 1 ? w[3] : w[2];
  return i & 2 ? hi : lo;
}

// kN elements in four 32-bit words; get and pick: element i (pick: i not known at compile time); raw: one
// element and masked ones in a word; wmax: the greater of two words, element by element; lift: the word
// with its -inf replaced by a value whose exponential is 0 (for f16, once it is fp32); count: n += the word's elements above those of `limit` (NaN is above everything).
template <int DT>
struct Elem;
template <>
struct Elem<FI_DTYPE_F32> {
  using T = float;
  static constexpr uint32_t kMasked = 0xFF800000u;  // -inf in every element
  static constexpr int kN = 4;
  __device__ static float get(const uint32_t (&w)[4], int i) { return __uint_as_float(w[i]); }
  __device__ static float pick(const uint32_t (&w)[4], int i) { return __uint_as_float(word_of(w, i)); }
  __device__ static float one(const void* p, int64_t i) { return static_cast<const float*>(p)[i]; }
  __device__ static uint32_t raw(const void* p, int64_t i) { return static_cast<const uint32_t*>(p)[i]; }
  __device__ static uint32_t wmax(uint32_t a, uint32_t b) {
    return __float_as_uint(max_nan(__uint_as_float(a), __uint_as_float(b)));
  }
  __device__ static float top(uint32_t w) { return __uint_as_float(w); }
  __device__ static uint32_t lift(uint32_t w) { return wmax(w, __float_as_uint(kFloor)); }
  __device__ static uint32_t spread(float x) { return __float_as_uint(x); }
  __device__ static uint32_t before(float x) { return __float_as_uint(below(x)); }
  __device__ static void count(uint32_t& n, uint32_t w, uint32_t limit) {
    n += !(__uint_as_float(w) <= __uint_as_float(limit)) ? 1 : 0;
  }
  __device__ static uint32_t counted(uint32_t n) { return n; }
};
template <>
struct Elem<FI_DTYPE_BF16> {
  using T = uint16_t;
  static constexpr uint32_t kMasked = 0xFF80FF80u;  // -inf in every element
  static constexpr int kN = 8;
  __device__ static float get(const uint32_t (&w)[4], int i) {
    return __uint_as_float(i & 1 ? w[i / 2] & 0xFFFF0000u : w[i / 2] << 16);
  }
  __device__ static float pick(const uint32_t (&w)[4], int i) {
    const uint32_t v = word_of(w, i >> 1);
    return __uint_as_float(i & 1 ? v & 0xFFFF0000u : v << 16);
  }
  __device__ static float one(const void* p, int64_t i) { return bf16_bits_to_f32(static_cast<const uint16_t*>(p)[i]); }
  __device__ static uint32_t raw(const void* p, int64_t i) {
    return (kMasked & 0xFFFF0000u) | static_cast<const uint16_t*>(p)[i];
  }
  __device__ static uint32_t wmax(uint32_t a, uint32_t b) { return max_bf16x2(a, b); }
  __device__ static float top(uint32_t w) {
    return max_nan(__uint_as_float(w << 16), __uint_as_float(w & 0xFFFF0000u));
  }
  // kFloor in bf16
  __device__ static uint32_t lift(uint32_t w) { return max_bf16x2(w, 0xCC80CC80u); }
  __device__ static uint32_t spread(float x) { return f32x2_to_bf16x2(x, x); }
  __device__ static uint32_t before(float x) {
    const uint32_t b = below16((uint16_t)f32_to_bf16_rn(x), 0xFF80u);
    return b | b << 16;
  }
  // greater or NaN: 1.0 each, added in bf16 (exact up to 256)
  __device__ static void count(uint32_t& n, uint32_t w, uint32_t limit) {
    asm("{\n .reg .b32 g;\n set.gtu.bf16x2.bf16x2 g, %1, %2;\n add.rn.bf16x2 %0, %0, g;\n}" : "+r"(n) : "r"(w), "r"(limit));
  }
  __device__ static uint32_t counted(uint32_t n) {
    return (uint32_t)(__uint_as_float(n << 16) + __uint_as_float(n & 0xFFFF0000u));
  }
};
template <>
struct Elem<FI_DTYPE_F16> {
  using T = uint16_t;
  static constexpr uint32_t kMasked = 0xFC00FC00u;  // -inf in every element
  static constexpr int kN = 8;
  __device__ static float get(const uint32_t (&w)[4], int i) {
    return i & 1 ? f16_hi_to_f32(w[i / 2]) : f16_lo_to_f32(w[i / 2]);
  }
  __device__ static float pick(const uint32_t (&w)[4], int i) {
    const uint32_t v = word_of(w, i >> 1);
    return f16_lo_to_f32(i & 1 ? v >> 16 : v);
  }
  __device__ static float one(const void* p, int64_t i) { return f16_lo_to_f32(static_cast<const uint16_t*>(p)[i]); }
  __device__ static uint32_t raw(const void* p, int64_t i) {
    return (kMasked & 0xFFFF0000u) | static_cast<const uint16_t*>(p)[i];
  }
  __device__ static uint32_t wmax(uint32_t a, uint32_t b) { return max_f16x2(a, b); }
  __device__ static float top(uint32_t w) { return max_nan(f16_lo_to_f32(w), f16_hi_to_f32(w)); }
  __device__ static uint32_t lift(uint32_t w) { return w; }
  __device__ static uint32_t spread(float x) { return f32x2_to_f16x2(x, x); }
  __device__ static uint32_t before(float x) {
    const uint32_t b = below16((uint16_t)f32_to_f16_rn(x), 0xFC00u);
    return b | b << 16;
  }
  __device__ static void count(uint32_t& n, uint32_t w, uint32_t limit) {
    asm("{\n .reg .b32 g;\n set.gtu.f16x2.f16x2 g, %1, %2;\n add.rn.f16x2 %0, %0, g;\n}" : "+r"(n) : "r"(w), "r"(limit));
  }
  __device__ static uint32_t counted(uint32_t n) { return (uint32_t)(f16_lo_to_f32(n) + f16_hi_to_f32(n)); }
};

// Sums relative to a reference point M = m log2 e (rounded to fp32, the same wherever it is
// formed from m): s = sum of 2^(z log2 e - M), t = sum of (z log2 e - M) times that.
struct Sums {
  float m, s, t;
};

__device__ __forceinline__ float point(float m) { return __fmul_rn(m, kLog2e); }

// The warp's 32 keys, one per lane, into ascending order by lane. (The loops stay loops: the
// kernel's time goes up with its code, as the instruction caches are small.)
template <typename T>
__device__ __forceinline__ T sort32(T v, int lane) {
#pragma unroll 1
  for (int size = 2; size <= 32; size *= 2) {
    const bool up = (lane & size) == 0 || size == 32;
#pragma unroll 1
    for (int o = size / 2; o > 0; o /= 2) {
      const T w = __shfl_xor_sync(0xffffffffu, v, o);
      v = (((lane & o) == 0) == up) == (v < w) ? v : w;
    }
  }
  return v;
}

// The 32 greatest of a descending list and an ascending one, descending.
template <typename T>
__device__ __forceinline__ T merge32(T list, T asc, int lane) {
  T v = list > asc ? list : asc;
#pragma unroll 1
  for (int o = 16; o > 0; o /= 2) {
    const T w = __shfl_xor_sync(0xffffffffu, v, o);
    v = ((lane & o) == 0) == (v > w) ? v : w;
  }
  return v;
}

__device__ __forceinline__ uint64_t ld_dsmem_u64(const void* p, uint32_t rank) {
  uint32_t remote;
  uint64_t v;
  asm("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(remote) : "r"(smem_addr(p)), "r"(rank));
  asm volatile("ld.shared::cluster.u64 %0, [%1];" : "=l"(v) : "r"(remote));
  return v;
}

template <int DT, int kThreads>
__global__ void __launch_bounds__(kThreads, kThreads == kFew ? 1 : 768 / kThreads)
    token_logprobs_kernel(const LogprobArgs p, int ctas) {
  using E = Elem<DT>;
  constexpr int kN = E::kN, kWarps = kThreads / 32;
  __shared__ uint64_t buffers[kWarps][kBuffer];
  __shared__ uint64_t lists[kWarps][32];
  __shared__ float sums[kWarps][3];
  __shared__ uint32_t before[kWarps], pending[kWarps];
  __shared__ uint32_t tops[kWarps][32];  // the threads' maxima, sorted by warps, or those of 32 groups of threads
  __shared__ struct {
    uint64_t list[32];
    float m, s, t;
    uint32_t before;
  } cta;
  const float kInf = __uint_as_float(0x7F800000u), kNan = __uint_as_float(0x7FC00000u);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int part = (int)(blockIdx.x % (unsigned)ctas);
  const int64_t row = blockIdx.x / (unsigned)ctas;
  const int K = p.topk;
  pdl_launch_dependents();
  pdl_wait();
  const typename E::T* z = static_cast<const typename E::T*>(p.logits) + row * p.ld;
  const int vocab = (int)p.vocab;
  // the row as `head` elements up to a 16-byte boundary, `vectors` of 16 bytes, and a tail; the
  // vectors in groups of kU per lane
  const int head = min(vocab, (int)((16 - (reinterpret_cast<uintptr_t>(z) & 15)) % 16 / sizeof(typename E::T)));
  const int vectors = (vocab - head) / kN;
  const uint4* const zv = reinterpret_cast<const uint4*>(z + head);
  const int groups = (vectors + 32 * kU - 1) / (32 * kU), step = ctas * kWarps;
  // a warp's groups in ascending order, then, for one warp of the row, the elements of both ends
  // (lanes 0 and 8 on, one each) as a group of their own
  const bool ends = part == 0 && warp == 0;
  const int first = part * kWarps + warp;
  const int mine = first < groups ? (groups - first + step - 1) / step : 0;
  const int rounds = mine + (ends ? 1 : 0);
  const int groups_all = groups / step + (groups % step >= (part + 1) * kWarps ? 1 : 0);  // that every warp here has
  // Groups come by asynchronous copies, kSlots - 1 of them ahead, into the warp's ring; a lane reads
  // what it copied itself, so it waits for nobody else.
  extern __shared__ __align__(16) uint8_t rings[];
  const uint32_t ring = smem_addr(rings) + (uint32_t)(warp * kSlots * kU * 32 + lane) * 16;
  const uint4* from = zv + (int64_t)first * 32 * kU + lane;  // of the next group
  int next_slot = 0;
  auto copy_group = [&](int round) {
    if (round < mine) {
#pragma unroll
      for (int u = 0; u < kU; ++u) {
        if (((first + round * step) * kU + u) * 32 + lane < vectors)
          asm volatile("cp.async.cg.shared.global.L2::256B [%0], [%1], 16;" ::"r"(
                           ring + (uint32_t)((next_slot * kU + u) * 32) * 16),
                       "l"(from + u * 32)
                       : "memory");
      }
      from += step * 32 * kU;
      next_slot = next_slot + 1 == kSlots ? 0 : next_slot + 1;
    }
    asm volatile("cp.async.commit_group;" ::: "memory");
  };
#pragma unroll
  for (int i = 0; i < kSlots - 1; ++i) copy_group(i);

  const int64_t token = p.tokens[row];
  const bool has_token = token >= 0 && token < p.vocab;
  const float zt = has_token ? E::one(z, token) : 0.0f;
  const int at_token = has_token ? (int)token : -1;
  const uint64_t token_key = has_token ? key_of(zt, (uint32_t)token) : 0;
  // behind the token a greater value comes before it, ahead of it an equal one too
  const uint32_t lim_behind = E::spread(zt), lim_ahead = E::before(zt);

  Sums a{kFloor, 0.0f, 0.0f};
  uint32_t earlier = 0;                 // entries before the token
  uint64_t list = 0;                    // this lane's entry of the warp's best, descending by lane
  uint32_t count = 0;                   // keys in the warp's buffer
  float above = K > 0 ? kNan : kInf;    // a value not above this cannot enter the list (NaN: any can)

#pragma unroll 1
  for (int round = 0; round < rounds; ++round) {
    uint32_t w[kU][4];
    int end_index = -1;  // this lane's element of an end
    if (round < mine) {
      asm volatile("cp.async.wait_group %0;" ::"n"(kSlots - 2) : "memory");
      const uint32_t at = ring + (uint32_t)(round % kSlots * kU * 32) * 16;
#pragma unroll
      for (int u = 0; u < kU; ++u)
        asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];"
                     : "=r"(w[u][0]), "=r"(w[u][1]), "=r"(w[u][2]), "=r"(w[u][3])
                     : "r"(at + u * 512));
      if ((first + round * step + 1) * (32 * kU) > vectors) {  // what is behind the last vector counts as masked
#pragma unroll
        for (int u = 0; u < kU; ++u)
#pragma unroll
          for (int i = 0; i < 4; ++i)
            w[u][i] = ((first + round * step) * kU + u) * 32 + lane < vectors ? w[u][i] : E::kMasked;
      }
    } else {
      const int tail = vocab - head - vectors * kN;
      if (lane < head && lane < 8) end_index = lane;
      if (lane >= 8 && lane - 8 < tail) end_index = vocab - tail + lane - 8;
#pragma unroll
      for (int u = 0; u < kU; ++u)
#pragma unroll
        for (int i = 0; i < 4; ++i) w[u][i] = E::kMasked;
      if (end_index >= 0) w[0][0] = E::raw(z, end_index);
    }
    copy_group(round + kSlots - 1);
    float mu[kU];  // the vectors' maxima
#pragma unroll
    for (int u = 0; u < kU; ++u)
      mu[u] = E::top(E::wmax(E::wmax(w[u][0], w[u][1]), E::wmax(w[u][2], w[u][3])));
    const float mx = max_nan(max_nan(mu[0], mu[1]), max_nan(mu[2], mu[3]));
    if (mx > a.m) {
      const float d = max_nan(point(a.m) - point(mx), kFar);
      const float c = exp2_fast(d);
      a.t = c * (a.t + d * a.s);
      a.s = c * a.s;
      a.m = mx;
    }
    // masked elements: an exponential of 0, or of 1 while the thread has seen nothing above
    // kFloor, which the first value above it, or another thread's, multiplies by 0
    const float minus = -point(a.m);
    const uint64_t minus_m = pack2(minus, minus), l2e = pack2(kLog2e, kLog2e);
    uint64_t s2 = pack2(a.s, 0.0f), t2 = pack2(a.t, 0.0f);
#pragma unroll
    for (int u = 0; u < kU; ++u) {
      uint32_t c[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) c[i] = E::lift(w[u][i]);
#pragma unroll
      for (int i = 0; i < kN; i += 2) {
        float x = E::get(c, i), y = E::get(c, i + 1);
        if (DT == FI_DTYPE_F16) {
          x = max_nan(x, kFloor);
          y = max_nan(y, kFloor);
        }
        const uint64_t d = fma2(pack2(x, y), l2e, minus_m);
        float ex, ey;
        unpack2(d, ex, ey);
        const uint64_t e = pack2(exp2_fast(ex), exp2_fast(ey));
        s2 = add2(s2, e);
        t2 = fma2(d, e, t2);
      }
    }
    float lo, hi;
    unpack2(s2, lo, hi);
    a.s = lo + hi;
    unpack2(t2, lo, hi);
    a.t = lo + hi;

    bool around = false;
    if (has_token) {
      // this lane's elements, first to last: all behind the token, all ahead of it, or around it
      const int low = round == mine ? max(end_index, 0) : head + ((first + round * step) * kU * 32 + lane) * kN;
      const int high = round == mine ? low + 1 : low + ((kU - 1) * 32 + 1) * kN;
      if (zt > -kInf && (at_token < low || at_token >= high)) {
        const uint32_t limit = at_token < low ? lim_behind : lim_ahead;
        uint32_t n = 0;
#pragma unroll
        for (int u = 0; u < kU; ++u)
#pragma unroll
          for (int i = 0; i < 4; ++i) E::count(n, w[u][i], limit);
        earlier += E::counted(n);
      } else {
        around = true;  // one by one, as for a token of NaN or -inf
      }
    }
    if (K > 0) {
      // Now and then, while every warp of the CTA still has a group: at least K elements are not
      // below the K-th of the threads' maxima, so that only a few more than K get past it. (Where
      // there are warps without a group, each warp takes its own lanes'.)
      if ((round == 0 || round == 1 || round == 3 || round == 7) && round < max(groups_all, 1)) {
        uint32_t v = a.m > kFloor ? order_of(a.m) : 0u;
        if (groups_all == 0) {
          v = __shfl_sync(0xffffffffu, sort32(v, lane), 32 - K);
        } else if (K <= kFewTops || kThreads == kFew) {
          // the same of the maxima of 32 groups of threads, in fewer steps. The first time all groups
          // are waited for; later their maxima are taken as they are, since an older maximum of a
          // group is an element as well.
          constexpr int kWidth = kThreads / 32;
#pragma unroll
          for (int o = 1; o < kWidth; o *= 2) v = max(v, __shfl_xor_sync(0xffffffffu, v, o));
          volatile uint32_t* const groups = tops[0];
          if ((lane & (kWidth - 1)) == 0) groups[threadIdx.x / kWidth] = v;
          if (round == 0)
            __syncthreads();
          else
            __syncwarp();
          uint32_t x = groups[lane];
          if (K <= kFewTops) {
            for (int k = 0; k < K; ++k) {  // (equal maxima count as one)
              v = __reduce_max_sync(0xffffffffu, x);
              x = x == v ? 0u : x;
            }
          } else {  // the least of those with fewer than K above
            int over = 0;
#pragma unroll
            for (int i = 0; i < 32; ++i) over += __shfl_sync(0xffffffffu, x, i) > x ? 1 : 0;
            v = __reduce_min_sync(0xffffffffu, over < K ? x : 0xFFFFFFFFu);
          }
        } else {
          v = sort32(v, lane);
          __syncthreads();
          tops[warp][31 - lane] = v;
          for (int o = kWarps / 2; o > 0; o >>= 1) {
            __syncthreads();
            if (warp < o) tops[warp][lane] = merge32(tops[warp][lane], tops[warp + o][31 - lane], lane);
          }
          __syncthreads();
          v = tops[0][K - 1];
        }
        const float b = below(value_of(v));
        if (b == b && !(b <= above)) above = b;
      }
      // the row's first elements come last here: of equal values they are the earlier ones
      if (round == mine) above = below(above);
    }
    if (__any_sync(0xffffffffu, around || !(mx <= above))) {
      uint32_t lists_us = 0;  // vectors to look at, for the list
#pragma unroll
      for (int u = 0; u < kU; ++u) lists_us |= __any_sync(0xffffffffu, !(mu[u] <= above)) ? 1u << u : 0u;
      uint32_t us = lists_us | (__any_sync(0xffffffffu, around) ? (1u << kU) - 1 : 0u);
#pragma unroll 1
      while (us) {
        const int u = __ffs(us) - 1;
        us &= us - 1;
        uint32_t v[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) v[i] = u < 2 ? (u == 0 ? w[0][i] : w[1][i]) : (u == 2 ? w[2][i] : w[3][i]);
        const int at = ((first + round * step) * kU + u) * 32 + lane;
        const int e0 = round == mine ? end_index : head + at * kN;
        const uint32_t valid = round == mine ? (u == 0 && end_index >= 0 ? 1u : 0u) : (at < vectors ? (1u << kN) - 1 : 0u);
        if (around) {
          if (zt != zt) {  // a NaN token: only a NaN of a lower index comes before it
#pragma unroll
            for (int i = 0; i < kN; ++i)
              earlier += (valid >> i & 1) && key_of(E::get(v, i), (uint32_t)(e0 + i)) > token_key ? 1 : 0;
          } else {
            uint32_t more = 0, same = 0;
#pragma unroll
            for (int i = 0; i < kN; ++i) {
              more |= !(E::get(v, i) <= zt) ? 1u << i : 0u;
              same |= E::get(v, i) == zt ? 1u << i : 0u;
            }
            const int ahead = at_token - e0;  // elements of this vector ahead of the token
            same &= ahead <= 0 ? 0u : (ahead >= kN ? ~0u : (1u << ahead) - 1);
            earlier += __popc((more | same) & valid);
          }
        }
        if (K > 0 && (lists_us >> u & 1)) {
          uint32_t todo = 0;
          // The limit of before this vector, and equal values too: what a merge on the way brings
          // into the list may have a higher index than an equal value still to come.
          const float from = below(above);
#pragma unroll
          for (int i = 0; i < kN; ++i) todo |= !(E::get(v, i) <= from) ? 1u << i : 0u;
          todo &= valid;
          for (uint32_t who; (who = __ballot_sync(0xffffffffu, todo != 0)) != 0; todo &= todo - 1) {
            const int i = __ffs(todo) - 1;  // this lane's next candidate
            if (todo) buffers[warp][count + __popc(who & ((1u << lane) - 1))] = key_of(E::pick(v, i), (uint32_t)(e0 + i));
            count += __popc(who);
            if (count >= 32) {
              __syncwarp();
              const uint64_t k = buffers[warp][lane];
              count -= 32;
              const uint64_t left = (uint32_t)lane < count ? buffers[warp][lane + 32] : 0;  // never beyond 63
              __syncwarp();
              buffers[warp][lane] = left;
              list = merge32(list, sort32(k, lane), lane);
              const uint64_t least = __shfl_sync(0xffffffffu, list, K - 1);
              if (least != 0) {
                const float own = value_of((uint32_t)(least >> 32));
                if (!(own <= above)) above = own;
              }
              __syncwarp();
            }
          }
        }
      }
    }
  }
  __syncwarp();
  // this lane's key of those still in the buffer (31 at most); their number, and 65536 if the warp has a list
  const uint64_t kept = (uint32_t)lane < count ? buffers[warp][lane] : 0;
  if (K > 0 && lane == 0) pending[warp] = count | (list != 0 ? 1u << 16 : 0u);
  // The sums and counts of the first `lanes` lanes (the others repeat them), in every lane: at the
  // greatest point of reference, so that one rescaling serves all.
  auto join_lanes = [&](int lanes) {
    const float m = value_of(__reduce_max_sync(0xffffffffu, order_of(a.m)));
    const float d = max_nan(point(a.m) - point(m), kFar), c = exp2_fast(d);
    a.t = c * (a.t + d * a.s);
    a.s = c * a.s;
    a.m = m;
    for (int o = lanes / 2; o > 0; o >>= 1) {
      a.s += __shfl_xor_sync(0xffffffffu, a.s, o);
      a.t += __shfl_xor_sync(0xffffffffu, a.t, o);
      earlier += __shfl_xor_sync(0xffffffffu, earlier, o);
    }
  };
  auto merge_lists = [&](int n) {  // the first n lists (a power of two), into warp 0's
    for (int o = n / 2; o > 0; o >>= 1) {
      __syncthreads();
      if (warp < o) {
        list = merge32(lists[warp][lane], lists[warp + o][31 - lane], lane);
        lists[warp][lane] = list;
      }
    }
  };
  join_lanes(32);
  if (lane == 0) {
    sums[warp][0] = a.m;
    sums[warp][1] = a.s;
    sums[warp][2] = a.t;
    before[warp] = earlier;
  }
  __syncthreads();
  if (K > 0) {
    // the warps' remaining keys, in a row, and 32 at a time into the lists
    uint64_t* const pool = &buffers[0][0];
    const uint32_t theirs = lane < kWarps ? pending[lane] : 0;
    const uint32_t all = __reduce_add_sync(0xffffffffu, theirs), keys = all & 0xFFFFu;
    const uint32_t at = __reduce_add_sync(0xffffffffu, lane < warp ? theirs & 0xFFFFu : 0u);
    if ((uint32_t)lane < count) pool[at + lane] = kept;
    __syncthreads();
    for (uint32_t c = warp * 32; c < keys; c += kWarps * 32)
      list = merge32(list, sort32(c + lane < keys ? pool[c + lane] : 0, lane), lane);
    lists[warp][lane] = list;
    int n = kWarps;  // lists that hold anything
    if (all < 1u << 16)
      while (n > 1 && (uint32_t)(n / 2) * 32 >= keys) n /= 2;
    merge_lists(n);
  }
  if (warp == 0) {
    const int w = lane % kWarps;
    a = Sums{sums[w][0], sums[w][1], sums[w][2]};
    earlier = before[w];
    join_lanes(kWarps);
  }
  if (ctas > 1) {
    if (warp == 0) {
      cta.list[lane] = list;
      if (lane == 0) {
        cta.m = a.m;
        cta.s = a.s;
        cta.t = a.t;
        cta.before = earlier;
      }
    }
    __syncwarp();
    cluster_sync();
    if (part == 0) {
      if (K > 0 && warp < ctas) lists[warp][lane] = ld_dsmem_u64(&cta.list[lane], (uint32_t)warp);
      if (warp == 0) {
        const uint32_t r = (uint32_t)(lane % ctas);
        a = Sums{__uint_as_float(ld_dsmem_u32(&cta.m, r)), __uint_as_float(ld_dsmem_u32(&cta.s, r)),
                 __uint_as_float(ld_dsmem_u32(&cta.t, r))};
        earlier = ld_dsmem_u32(&cta.before, r);
        join_lanes(ctas);
      }
    }
    __syncwarp();
    cluster_sync();  // no CTA leaves while its sums are read
    if (part != 0) return;
    if (K > 0) merge_lists(ctas);
  }
  __syncthreads();
  if (threadIdx.x == 0) {
    cta.m = a.m;
    cta.s = a.s;
    cta.t = a.t;
  }
  __syncthreads();
  a = Sums{cta.m, cta.s, cta.t};
  const bool far = !(fabsf(a.m) <= kFarMax);
  if (far) {
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
  // The point is off m log2 e by its rounding, `off`, and every exponential by the power of two of that
  // (of a far row the sums are relative to the maximum itself, t in natural units). s is divided by the
  // maximum's own exponential, as the loop found it: s holds it, so the quotient is 1 at least and just
  // that where the other entries add nothing, and its logarithm 0. With t's true value at most 0, no log
  // probability comes out above 0 and no entropy below, and a row with one entry left has 0 for both.
  const float off = far ? 0.0f : fmaf(a.m, kLog2e, -point(a.m));
  const float ln_sum = empty ? 0.0f : logf(a.s / exp2_fast(off));
  const float t = __fsub_rn(a.t, __fmul_rn(off, a.s));
  const float mean = empty ? 0.0f : (t > 0.0f ? 0.0f : t) / a.s * (far ? 1.0f : kLn2);
  auto logprob_of = [&](float x) { return empty ? x : (x - a.m) - ln_sum; };
  if (lane == 0) {
    p.logprob[row] = has_token ? logprob_of(zt) : __uint_as_float(0x7FC00000u);
    p.entropy[row] = ln_sum - mean;
    p.rank[row] = has_token ? (int64_t)earlier : -1;
  }
  if (lane < K) {
    p.top_logprobs[row * K + lane] = logprob_of(value_of((uint32_t)(list >> 32)));
    p.top_ids[row * K + lane] = (int64_t)(uint32_t)~(uint32_t)list;
  }
}

template <int DT, int kThreads>
int launch(const LogprobArgs& a, int ctas, cudaStream_t stream) {
  constexpr int kRings = kThreads * kSlots * kU * 16;
  static_assert(kRings <= 192 * 1024, "beside the lists in shared memory");
  static std::atomic<bool> configured[kMaxDevices];
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= kMaxDevices) return set_cuda_error("cudaGetDevice");
  if (!configured[dev]) {
    if (cudaFuncSetAttribute(token_logprobs_kernel<DT, kThreads>, cudaFuncAttributeMaxDynamicSharedMemorySize, kRings) !=
        cudaSuccess)
      return set_cuda_error("cudaFuncSetAttribute(token_logprobs_kernel)");
    configured[dev] = true;
  }
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
  cfg.dynamicSmemBytes = kRings;
  cfg.stream = stream;
  cfg.attrs = attr;
  cfg.numAttrs = 2;
  if (cudaLaunchKernelEx(&cfg, token_logprobs_kernel<DT, kThreads>, a, ctas) != cudaSuccess)
    return set_cuda_error("token_logprobs_kernel launch");
  return FI_OK;
}

template <int DT>
int launch_rows(const LogprobArgs& a, cudaStream_t stream) {
  // CTAs per row: as many as leave each a group of vectors for most of its warps, while the rows alone
  // do not give every SM its CTAs.
  const int64_t groups = a.vocab / Elem<DT>::kN / 128, sms = device_sm_count();
  // Few rows: large CTAs where the lists' limits are worth more threads. Measured (us, 256 threads /
  // 1024): 33 bf16 rows of 100000 with 5 alternatives 11.2 / 10.0, with 20 15.2 / 11.4, fp32 17.0 / 13.5;
  // 100 rows with 20 19.3 / 17.0, with 5 14.4 / 14.3; one row of 152064 with 5 8.9 / 10.9,
  // fp32 9.7 / 10.9, of 260000 12.1 / 11.4.
  const bool few = a.topk > kFewTops ? a.rows <= sms && groups >= 64
                                     : (a.rows * 16 <= sms ? groups >= 400 : a.topk > 0 && a.rows * 4 <= sms && groups >= 64);
  // Many rows: with small CTAs fewer warps wait at a row's start and end, with large ones the last
  // wave is shorter and the lists' limits come from more threads. Measured with 128 / 256 threads
  // (us): 4096 rows of 32000 with 5 alternatives 89 / 107, of 5001 38 / 65, 1000 of 5000 with 20 17.4 /
  // 25.4, 2047 of 152064 without a list 99 / 111, with 32 217 / 212, 3600 of
  // 100000 with 20 234 / 263; 1024 fp32 rows of 152064 with 5 135 / 122, 3600 of 25000 85 / 101.
  const int64_t small = 768 / kShort * sms, large = 768 / kMany * sms;  // CTAs that the device holds
  const bool fewer_waves = (a.rows + small - 1) / small * small * 100 <= (a.rows + large - 1) / large * large * 118;
  if (a.rows > large && (groups < 32 || (a.topk == 0 ? a.rows >= 8 * sms : fewer_waves)))
    return launch<DT, kShort>(a, 1, stream);
  const int64_t warps = (few ? kFew : kMany) / 32, slots = few ? sms : large;
  int ctas = 1;
  static_assert(kMany / 32 >= kMaxCtas && kFew / 32 >= kMaxCtas, "a warp takes the list of each CTA of a cluster");
  while (ctas < kMaxCtas && a.rows * ctas * 2 <= slots && groups >= ctas * warps + 4) ctas *= 2;
  return few ? launch<DT, kFew>(a, ctas, stream) : launch<DT, kMany>(a, ctas, stream);
}

}  // namespace

int launch_token_logprobs(const LogprobArgs& a, int dtype, cudaStream_t stream) {
  switch (dtype) {
    case FI_DTYPE_BF16:
      return launch_rows<FI_DTYPE_BF16>(a, stream);
    case FI_DTYPE_F16:
      return launch_rows<FI_DTYPE_F16>(a, stream);
    default:
      return launch_rows<FI_DTYPE_F32>(a, stream);
  }
}

}  // namespace fi
