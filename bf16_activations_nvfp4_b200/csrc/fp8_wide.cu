// 8-bit products with a scale per block of 128 at prompt sizes (sm_100a: tcgen05 on CTA pairs).
//
// The same sums as fp8_mm.cu, for many activation rows, where the tensor cores are the bound. A
// pair of CTAs (a cluster of 2) owns a tile of 256 activation rows x 256 weight rows, or of 256
// activation rows x (128 gate + 128 up rows) in the gated form: one tcgen05.mma of both SMs reads
// 128 rows of A from each CTA and 128 rows of B from each, so a CTA loads 32 KB per 128 k and
// feeds 256 columns. Roles of a CTA (12 warps):
//   warp 0      TMA producer of its 128 A rows and 128 B rows into a ring of 5 stages; the bytes of
//               both CTAs complete one barrier, in the pair's first CTA;
//   warp 1      in the first CTA, one thread issues the MMAs for both; the commits arrive in both;
//   warps 2-3   the scales As * Ws of a block, up to 16 blocks ahead, into a ring;
//   warps 4-11  epilogue, one thread per activation row and half of the columns (128): a block's
//               sums, times the row's scale, are added to 128 fp32 registers while the tensor
//               cores fill the other TMEM buffer. setmaxnreg gives these warps 216 registers. A
//               warp takes 64 columns of each half, so that in the gated form a thread has the
//               gates and their up columns.
// The CTAs are persistent: tiles go round-robin over the pairs, in groups of 8 along m, so that
// the pairs at work share operand rows in L2; the next tile's blocks start while the last one's
// outputs are written.
//
// Bound by the chain of a block's steps (MMAs, commit, TMEM loads, additions, release: two TMEM
// buffers are in flight) and, under sustained load, by power: 720 to 750 cycles per block of a pair
// where the MMAs and loads alone take 638 and the nominal rate is 512. 8192 x 4096 x 14336 takes
// 404 us (2.4 PFLOP/s), 470 at the power limit; 4096 rows of the gated 2 x 17408 x 5120 617 us, 730
// at the power limit. N = 128 instructions with four buffers took 646 us on the former where this form took 504, 16
// epilogue warps 559 against 450.
//
// Every wait is bounded; on a timeout the roles stop and every thread still meets the barriers.
#include <cstdint>
#include <algorithm>
#include <atomic>

#include "fp8_tc.cuh"

namespace fi {

namespace {

constexpr int kStages = 5, kBufs = 2, kThreads = 384;
constexpr int kGroup = 8, kGroups = 2;                          // blocks of k whose scales share a barrier; groups in the ring
constexpr int kRows = 128;                                      // activation rows of a CTA
constexpr uint32_t kHalfBytes = kRows * 128, kStageBytes = 2 * kHalfBytes;
constexpr uint32_t kPairBytes = 2 * kStageBytes;                // bytes a full barrier waits for
constexpr uint32_t kOutBytes = 32 * 1024;                       // staging of the epilogue: 4 KB per warp
constexpr uint32_t kScaleBytes = kGroups * kGroup * 2 * kRows * 4;
constexpr uint32_t kBarBytes = (2 * kStages + kBufs + 2 * kGroups + 1) * 8;
constexpr int kGroupM = 8;  // 4, 12, 16 and 32 are within 3%
constexpr uint32_t kSmem = 1024 + kStages * kStageBytes + kOutBytes + kScaleBytes + kBarBytes;
static_assert(kBufs <= kStages, "an epilogue that is behind sees each block's barrier before its next phase is over");
static_assert(32 * 128 <= kOutBytes / 8, "a warp stages 128 bytes of 32 rows");
constexpr int kEpiRegs = 216, kOtherRegs = 64;
// registers after the split: the epilogue's two warpgroups and the other one stay within the launch's 168 a thread
static_assert(256 * kEpiRegs + 128 * kOtherRegs <= kThreads * 168, "register split");

__device__ __forceinline__ uint32_t cluster_rank() {
  uint32_t r;
  asm("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
  return r;
}

// This shared-memory address in the cluster's CTA `rank`.
__device__ __forceinline__ uint32_t map_to(uint32_t addr, uint32_t rank) {
  uint32_t r;
  asm("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(r) : "r"(addr), "r"(rank));
  return r;
}

__device__ __forceinline__ void tma_load_pair(uint32_t dst, const CUtensorMap* map, int x, int y, uint32_t bar) {
  asm volatile(
      "cp.async.bulk.tensor.2d.cta_group::2.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3}], "
      "[%4];" ::"r"(dst),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(x), "r"(y), "r"(bar)
      : "memory");
}

__device__ __forceinline__ void umma_f8_pair(uint32_t d_tmem, uint64_t adesc, uint64_t bdesc, uint32_t idesc,
                                             uint32_t accumulate) {
  asm volatile(
      "{\n .reg .pred p;\n setp.ne.b32 p, %4, 0;\n tcgen05.mma.cta_group::2.kind::f8f6f4 [%0], %1, %2, %3, p;\n}" ::"r"(
          d_tmem),
      "l"(adesc), "l"(bdesc), "r"(idesc), "r"(accumulate)
      : "memory");
}

// Arrives on the barrier at this offset in both CTAs when the MMAs issued so far are complete.
__device__ __forceinline__ void umma_commit_pair(uint64_t* bar) {
  asm volatile(
      "tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64 [%0], %1;" ::"r"(
          smem_addr(bar)),
      "h"((uint16_t)3)
      : "memory");
}

// Arrives on a barrier of the pair. It orders TMEM reads only (a tcgen05 fence precedes it), so the
// default scope is enough: at cluster scope each arrival is a memory barrier, and the kernel ran at
// half its speed.
__device__ __forceinline__ void mbar_arrive_remote_if(uint32_t yes, uint32_t addr) {
  asm volatile(
      "{\n .reg .pred p;\n setp.ne.b32 p, %0, 0;\n @p mbarrier.arrive.shared::cluster.b64 _, [%1];\n}" ::"r"(yes),
      "r"(addr)
      : "memory");
}

// Keeps uses of registers that an earlier tmem_wait_ld covered below it.
__device__ __forceinline__ void tmem_pass32(uint32_t (&r)[32]) {
  asm volatile(""
               : "+r"(r[0]), "+r"(r[1]), "+r"(r[2]), "+r"(r[3]), "+r"(r[4]), "+r"(r[5]), "+r"(r[6]), "+r"(r[7]),
                 "+r"(r[8]), "+r"(r[9]), "+r"(r[10]), "+r"(r[11]), "+r"(r[12]), "+r"(r[13]), "+r"(r[14]), "+r"(r[15]),
                 "+r"(r[16]), "+r"(r[17]), "+r"(r[18]), "+r"(r[19]), "+r"(r[20]), "+r"(r[21]), "+r"(r[22]),
                 "+r"(r[23]), "+r"(r[24]), "+r"(r[25]), "+r"(r[26]), "+r"(r[27]), "+r"(r[28]), "+r"(r[29]),
                 "+r"(r[30]), "+r"(r[31])
               :
               : "memory");
}

// (x, y) += (a, b) * s, both lanes of one packed instruction.
__device__ __forceinline__ void fma_pair(float& x, float& y, uint32_t a, uint32_t b, float s) {
  asm("{\n .reg .b64 d, e, f;\n mov.b64 d, {%2, %3};\n mov.b64 e, {%4, %4};\n mov.b64 f, {%0, %1};\n"
      " fma.rn.f32x2 f, d, e, f;\n mov.b64 {%0, %1}, f;\n}"
      : "+f"(x), "+f"(y)
      : "r"(a), "r"(b), "f"(s));
}

struct WideArgs {
  Fp8MmArgs p;
  int tiles_n;        // tiles along n (256 columns, or 128 of the gated form)
  int64_t tiles;      // tiles in all
  int wide_stores;    // out rows take 16-byte stores
};

// The tile's (m, n) in units of tiles.
__device__ __forceinline__ void tile_at(const WideArgs& w, int64_t t, int& tm, int& tn) {
  const int64_t per = (int64_t)kGroupM * w.tiles_n;
  const int g = (int)(t / per);
  const int r = (int)(t - g * per);
  const int gm = min(kGroupM, w.p.tiles_m - g * kGroupM);
  tn = r / gm;
  tm = g * kGroupM + (r - tn * gm);
}

// One warp's 32 rows x 64 columns of `acc` (from C0 on) to out rows row0.., columns col0..: through
// 4 KB of shared memory, so that 128 bytes of a row leave together. Runs once per tile, so what
// counts is that it is short: its instructions come from far.
template <int C0, int OUT>
__device__ __forceinline__ void store_rows(const Fp8MmArgs& p, bool wide, const float (&acc)[128], uint8_t* stage,
                                           int lane, int64_t row0, int64_t col0) {
  constexpr int es = OUT == FI_DTYPE_F32 ? 4 : 2, per = 16 / es;  // elements per 16 bytes
  const uint32_t sbase = smem_addr(stage);
  const int64_t pitch = p.n * es;
  // 16-byte piece ch of row r; the rows' pieces are permuted so that no two lanes meet in a bank
  auto piece = [&](int r, int ch) { return sbase + (uint32_t)(r * 128 + ((ch ^ (r & 7)) * 16)); };
  constexpr int kStep = 8 * per;  // columns of 128 bytes
#pragma unroll
  for (int c = 0; c < 64; c += kStep) {
#pragma unroll
    for (int ch = 0; ch < 8; ++ch) {
      const float* a = acc + C0 + c + ch * per;
      uint32_t w[4];
#pragma unroll
      for (int i = 0; i < 4; ++i)
        w[i] = OUT == FI_DTYPE_F32 ? __float_as_uint(a[i])
                                   : (OUT == FI_DTYPE_F16 ? f32x2_to_f16x2(a[2 * i % 8], a[(2 * i + 1) % 8])
                                                          : f32x2_to_bf16x2(a[2 * i % 8], a[(2 * i + 1) % 8]));
      asm volatile("st.shared.v4.u32 [%0], {%1, %2, %3, %4};" ::"r"(piece(lane, ch)), "r"(w[0]), "r"(w[1]), "r"(w[2]),
                   "r"(w[3])
                   : "memory");
    }
    __syncwarp();
    if (wide && row0 + 32 <= p.m && col0 + c + kStep <= p.n) {
      uint8_t* dst = static_cast<uint8_t*>(p.out) + (row0 + lane / 8) * pitch + (col0 + c + (lane % 8) * per) * es;
#pragma unroll 1
      for (int r = lane / 8; r < 32; r += 4) {
        uint4 v;
        asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];"
                     : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
                     : "r"(piece(r, lane % 8)));
        *reinterpret_cast<uint4*>(dst) = v;
        dst += 4 * pitch;
      }
    } else {
      // rows of any pitch: a row's 128 bytes by all lanes, a word each, so that neighbouring lanes
      // write neighbouring addresses. A word whose address is odd to it goes as two halves. (Element by
      // element in the order above: 339 x 12610 x 2480 to f16 52 us.)
      const int rows = (int)min((int64_t)32, p.m - row0);
      const int64_t col = col0 + c + lane * (4 / es);
      uint8_t* dst = static_cast<uint8_t*>(p.out) + row0 * pitch + col * es;
      const bool words = es == 4 || (p.n % 2 == 0 && (reinterpret_cast<uintptr_t>(p.out) & 3) == 0);
#pragma unroll 4
      for (int r = 0; r < rows; ++r) {
        uint32_t v;
        asm volatile("ld.shared.u32 %0, [%1];" : "=r"(v) : "r"(piece(r, lane / 4) + (uint32_t)(lane % 4) * 4));
        if (words) {
          if (col < p.n) *reinterpret_cast<uint32_t*>(dst) = v;
        } else {
          if (col < p.n) *reinterpret_cast<uint16_t*>(dst) = (uint16_t)v;
          if (col + 1 < p.n) *reinterpret_cast<uint16_t*>(dst + 2) = (uint16_t)(v >> 16);
        }
        dst += pitch;
      }
    }
    __syncwarp();
  }
}

template <bool GATED, int OUT>
__global__ void __launch_bounds__(kThreads, 1)
    fp8_wide_kernel(const WideArgs w, const __grid_constant__ CUtensorMap tmap_a,
                    const __grid_constant__ CUtensorMap tmap_w0, const __grid_constant__ CUtensorMap tmap_w1) {
  const Fp8MmArgs& p = w.p;
  extern __shared__ __align__(1024) uint8_t smem_raw[];
  __shared__ volatile int abort_flag;
  __shared__ uint32_t tmem_slot;
  const uint32_t raw_s = smem_addr(smem_raw);
  const uint32_t base = (raw_s + 1023u) & ~1023u;
  uint8_t* const basep = smem_raw + (base - raw_s);
  uint8_t* const staging = basep + kStages * kStageBytes;
  float* const scales = reinterpret_cast<float*>(staging + kOutBytes);  // [group][block][row][column half]
  uint64_t* const full = reinterpret_cast<uint64_t*>(staging + kOutBytes + kScaleBytes);
  // a block's MMAs are complete: its stage may be refilled and its sums read (one commit for both)
  uint64_t* const done = full + kStages;
  uint64_t* const tmem_empty = done + kStages;
  uint64_t* const scale_full = tmem_empty + kBufs;
  uint64_t* const scale_empty = scale_full + kGroups;
  uint64_t* const drain = scale_empty + kGroups;

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int rank = (int)cluster_rank();
  const int64_t pair = blockIdx.x >> 1, pairs = gridDim.x >> 1;
  const int64_t my_tiles = pair < w.tiles ? (w.tiles - pair + pairs - 1) / pairs : 0;
  const int KB = p.kblocks;

  if (threadIdx.x == 0) {
    abort_flag = 0;
    for (int i = 0; i < kStages; ++i) {
      mbar_init(&full[i], 1);
      mbar_init(&done[i], 1);
    }
    for (int i = 0; i < kBufs; ++i) {
      mbar_init(&tmem_empty[i], 16);  // the epilogue warps of both CTAs
    }
    for (int i = 0; i < kGroups; ++i) {
      mbar_init(&scale_full[i], 2);
      mbar_init(&scale_empty[i], 8);
    }
    mbar_init(drain, 1);
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
  }
  if (warp == 1) {
    asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_addr(&tmem_slot)),
                 "r"(512u)
                 : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;" ::: "memory");
  }
  asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory");
  __syncthreads();
  cluster_sync();  // both CTAs' barriers exist
  asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
  const uint32_t tmem = tmem_slot;
  pdl_launch_dependents();

  if (warp < 4) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kOtherRegs));
    if (warp == 0) {
      if (lane == 0) {
        pdl_wait();
        const uint32_t full0 = map_to(smem_addr(full), 0);
        const CUtensorMap* const bmap = GATED && rank == 1 ? &tmap_w1 : &tmap_w0;
        int st = 0;
        uint32_t phase = 0;   // of the stage's round: the first has nothing to wait for
        bool first = true, ok = true;
        int64_t issued = 0;
        for (int64_t t = 0; t < my_tiles && ok && !p.debug_stall; ++t) {
          int tm, tn;
          tile_at(w, pair + t * pairs, tm, tn);
          const int ya = (tm * 2 + rank) * kRows, yb = GATED ? tn * 128 : (tn * 2 + rank) * 128;
          for (int i = 0; i < KB; ++i) {
            if (!first &&
                !mbar_wait_spin(&done[st], phase ^ 1, &abort_flag, p.timeout_ns, p.err, 2u)) {
              ok = false;
              break;
            }
            const uint32_t dst = base + (uint32_t)st * kStageBytes, bar = full0 + (uint32_t)st * 8;
            if (rank == 0) mbar_arrive_expect_tx(&full[st], kPairBytes);
            tma_load_pair(dst, &tmap_a, i * kFp8Block, ya, bar);
            tma_load_pair(dst + kHalfBytes, bmap, i * kFp8Block, yb, bar);
            ++issued;
            if (++st == kStages) {
              st = 0;
              phase ^= 1;
              first = false;
            }
          }
        }
        if (rank == 0) {  // both CTAs' copies in flight land before either gives its memory up
          volatile int never = 0;
          for (int64_t i = issued > kStages ? issued - kStages : 0; i < issued; ++i)
            mbar_wait_spin(&full[i % kStages], (uint32_t)(i / kStages) & 1, &never, p.timeout_ns, p.err, 4u);
        }
      }
      __syncwarp();
    } else if (warp == 1) {
      if (lane == 0 && rank == 0) {
        constexpr uint32_t idesc = f8_idesc(256, 256);
        pdl_wait();  // the limit of a wait counts from the preceding kernel's end
        const int64_t total = my_tiles * KB;
        int st = 0;
        uint32_t phase = 0;
        bool ok = true;
        for (int64_t it = 0; it < total; ++it) {
          const uint32_t b = (uint32_t)it & 1;
          ok = mbar_wait_spin(&full[st], phase, &abort_flag, p.timeout_ns, p.err, 1u) &&
               (it < kBufs || mbar_wait_spin(&tmem_empty[b], ((uint32_t)it / kBufs - 1) & 1, &abort_flag,
                                             p.timeout_ns, p.err, 1u));
          if (!ok) break;
          asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
          const uint64_t adesc = sw128_desc(base + (uint32_t)st * kStageBytes);
          const uint64_t bdesc = sw128_desc(base + (uint32_t)st * kStageBytes + kHalfBytes);
#pragma unroll
          for (int s = 0; s < 4; ++s)  // K = 32 bytes each
            umma_f8_pair(tmem + b * 256, adesc + (uint64_t)(2 * s), bdesc + (uint64_t)(2 * s), idesc, s > 0);
          umma_commit_pair(&done[st]);
          if (++st == kStages) {
            st = 0;
            phase ^= 1;
          }
        }
        if (!ok) {  // the MMAs in flight end before TMEM is freed
          volatile int never = 0;
          umma_commit_pair(drain);
          mbar_wait_spin(drain, 0, &never, p.timeout_ns, p.err, 8u);
        }
      }
      __syncwarp();
    } else {
      // warps 2 and 3: 64 rows each, two per lane; four blocks are loaded while the four before
      // them are multiplied and stored
      pdl_wait();
      constexpr int kBatch = 4;
      const int r0 = (warp - 2) * 64 + lane;
      const int64_t wblocks = (p.n + kFp8Block - 1) / kFp8Block;
      float* const dst0 = scales + r0 * 2;
      float next[kBatch][4];
      uint32_t it = 0, g = 0, phase = 1;  // blocks so far, the group, its barrier's phase
      bool ok = true;
      for (int64_t t = 0; t < my_tiles && ok; ++t) {
        int tm, tn;
        tile_at(w, pair + t * pairs, tm, tn);
        const int64_t row = ((int64_t)tm * 2 + rank) * kRows + r0;
        const int64_t blk = GATED ? tn : (int64_t)tn * 2;
        const bool in0 = row < p.m, in1 = row + 32 < p.m, win1 = GATED || blk + 1 < wblocks;
        const float* const a0 = p.As + (in0 ? row : 0) * KB;
        const float* const a1 = p.As + (in1 ? row + 32 : 0) * KB;
        const float* const w0 = p.Ws[0] + blk * KB;
        const float* const w1 = GATED ? p.Ws[1] + blk * KB : p.Ws[0] + (win1 ? blk + 1 : 0) * KB;
        auto load = [&](int i0) {
#pragma unroll
          for (int d = 0; d < kBatch; ++d) {
            if (i0 + d < KB) {
              next[d][0] = __ldg(a0 + i0 + d);
              next[d][1] = __ldg(a1 + i0 + d);
              next[d][2] = __ldg(w0 + i0 + d);
              next[d][3] = __ldg(w1 + i0 + d);
            }
          }
        };
        load(0);
        for (int i0 = 0; i0 < KB && ok; i0 += kBatch) {
          float v[kBatch][4];
#pragma unroll
          for (int d = 0; d < kBatch; ++d) {
            v[d][0] = in0 ? next[d][0] : 0.0f;
            v[d][1] = in1 ? next[d][1] : 0.0f;
            v[d][2] = next[d][2];
            v[d][3] = win1 ? next[d][3] : 0.0f;
          }
          load(i0 + kBatch);
#pragma unroll
          for (int d = 0; d < kBatch; ++d) {
            if (i0 + d < KB && ok) {
              if (it % kGroup == 0 && it >= kGroup * kGroups) {
                ok = mbar_wait_spin(&scale_empty[g], phase, &abort_flag, p.timeout_ns, p.err, 2u);
                ok = __all_sync(0xffffffffu, ok);
              }
              float2* const dst = reinterpret_cast<float2*>(dst0 + it % (kGroup * kGroups) * (2 * kRows));
              dst[0] = make_float2(v[d][0] * v[d][2], v[d][0] * v[d][3]);
              dst[32] = make_float2(v[d][1] * v[d][2], v[d][1] * v[d][3]);
              if (++it % kGroup == 0 || (t + 1 == my_tiles && i0 + d + 1 == KB)) {
                __syncwarp();
                if (lane == 0) mbar_arrive(&scale_full[g]);
                if (++g == kGroups) {
                  g = 0;
                  phase ^= 1;
                }
              }
            }
          }
        }
      }
    }
  } else {
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kEpiRegs));
    pdl_wait();  // before the first wait with a limit, and before any output is written
    const int epi = warp - 4, quarter = warp & 3, half = epi >> 2;
    uint8_t* const stage = staging + epi * (kOutBytes / 8);
    const uint32_t empty0 = map_to(smem_addr(tmem_empty), 0);
    // A wait that runs out raises the abort flag; the ones after it then give up at once, and the
    // blocks' sums are what TMEM held: the way out is between tiles.
    const uint32_t done0 = smem_addr(done), done_end = done0 + kStages * 8;
    const uint32_t sp0 = smem_addr(scales) + (uint32_t)(quarter * 32 + lane) * 8;
    const uint32_t lanes = tmem + ((uint32_t)(quarter * 32) << 16) + (uint32_t)(half * 64);
    const uint32_t first = lane == 0;
    uint32_t done_bar = done0, phase = 0;  // the next block's barrier and its phase
    uint32_t it = 0;                       // blocks so far (its low bits count)
    float s0, s1;                          // the scales of the next block
    auto load_scales = [&](uint32_t i) {
      if (i % kGroup == 0)
        mbar_wait_spin(&scale_full[i / kGroup % kGroups], i / (kGroup * kGroups) & 1, &abort_flag, p.timeout_ns, p.err,
                       16u);
      asm volatile("ld.shared.v2.f32 {%0, %1}, [%2];"
                   : "=f"(s0), "=f"(s1)
                   : "r"(sp0 + i % (kGroup * kGroups) * (2 * kRows * 4)));
    };
    for (int64_t t = 0; t < my_tiles && !__any_sync(0xffffffffu, abort_flag != 0); ++t) {
      float acc[128];
#pragma unroll
      for (int c = 0; c < 128; ++c) acc[c] = 0.0f;
      load_scales(it);
#pragma unroll 1
      for (int i = 0; i < KB; ++i) {
        mbar_wait_addr(done_bar, phase, &abort_flag, p.timeout_ns, p.err, 16u);
        __syncwarp();
        asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
        done_bar += 8;
        if (done_bar == done_end) {
          done_bar = done0;
          phase ^= 1;
        }
        const uint32_t b = it & 1, taddr = lanes + b * 256;
        const float c0 = s0, c1 = s1;
        // 64 columns at a time in two loads: the buffer is held for two load latencies
        uint32_t d0[32], d1[32];
        tmem_ld_async(taddr, d0);
        tmem_ld_async(taddr + 32, d1);
        tmem_wait_ld(d0);
        tmem_pass32(d1);
#pragma unroll
        for (int q = 0; q < 32; q += 2) fma_pair(acc[q], acc[q + 1], d0[q], d0[q + 1], c0);
        tmem_ld_async(taddr + 128, d0);
#pragma unroll
        for (int q = 0; q < 32; q += 2) fma_pair(acc[32 + q], acc[33 + q], d1[q], d1[q + 1], c0);
        tmem_ld_async(taddr + 160, d1);
        tmem_wait_ld(d0);
        tmem_pass32(d1);
        // everything is in registers: the buffer, and at a group's end its scales, are free
        asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory");
        __syncwarp();
        mbar_arrive_remote_if(first, empty0 + b * 8);
        // the next block's scales are read while this one's columns are added
        if (i + 1 < KB) load_scales(it + 1);
        if (it % kGroup == kGroup - 1 && first) mbar_arrive(&scale_empty[it / kGroup % kGroups]);
        ++it;
#pragma unroll
        for (int q = 0; q < 32; q += 2) fma_pair(acc[64 + q], acc[65 + q], d0[q], d0[q + 1], c1);
#pragma unroll
        for (int q = 0; q < 32; q += 2) fma_pair(acc[96 + q], acc[97 + q], d1[q], d1[q + 1], c1);
      }
      if (!__any_sync(0xffffffffu, abort_flag != 0)) {
        int tm, tn;
        tile_at(w, pair + t * pairs, tm, tn);
        const int64_t row0 = ((int64_t)tm * 2 + rank) * kRows + quarter * 32;
        if (GATED) {  // the first 64 columns are gates, the others their up columns
#pragma unroll
          for (int c = 0; c < 64; c += 2) silu_times(acc[c], acc[c + 1], acc[64 + c], acc[65 + c]);
          store_rows<0, OUT>(p, w.wide_stores != 0, acc, stage, lane, row0, (int64_t)tn * 128 + half * 64);
        } else {
          store_rows<0, OUT>(p, w.wide_stores != 0, acc, stage, lane, row0, (int64_t)tn * 256 + half * 64);
          store_rows<64, OUT>(p, w.wide_stores != 0, acc, stage, lane, row0, (int64_t)tn * 256 + 128 + half * 64);
        }
      }
    }
  }

  asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory");
  __syncthreads();
  cluster_sync();  // neither CTA leaves while the other's MMAs or arrivals may reach it
  if (warp == 1) {
    asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
    asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(512u) : "memory");
  }
}

}  // namespace

int launch_fp8_wide(Fp8MmArgs a, bool gated, cudaStream_t stream) {
  WideArgs w;
  w.p = a;
  const int64_t tiles_m = (a.m + 255) / 256, tiles_n = gated ? (a.n + 127) / 128 : (a.n + 255) / 256;
  if (a.n > 0x7ffffe00LL || a.m > 0x7ffffe00LL || a.k > 0x7fffff00LL)
    return set_error(FI_ERR_UNSUPPORTED_SHAPE, "m=%lld n=%lld k=%lld is too large", (long long)a.m, (long long)a.n,
                     (long long)a.k);
  w.p.tiles_m = (int)tiles_m;
  w.p.splits = 1;
  w.tiles_n = (int)tiles_n;
  w.tiles = tiles_m * tiles_n;
  w.wide_stores = (reinterpret_cast<uintptr_t>(a.out) & 15) == 0 && a.n * (a.out_dtype == FI_DTYPE_F32 ? 4 : 2) % 16 == 0;
  CUtensorMap ta, tw[2];
  int rc = encode_codes(&ta, a.A, a.k, a.m, kRows);
  for (int t = 0; t < (gated ? 2 : 1) && rc == FI_OK; ++t) rc = encode_codes(&tw[t], a.W[t], a.k, a.n, 128);
  if (rc != FI_OK) return rc;
  if (!gated) tw[1] = tw[0];
  const int out = a.out_dtype;
  auto pick = [&](auto g) {
    constexpr bool kGated = decltype(g)::value;
    return out == FI_DTYPE_BF16  ? fp8_wide_kernel<kGated, FI_DTYPE_BF16>
           : out == FI_DTYPE_F16 ? fp8_wide_kernel<kGated, FI_DTYPE_F16>
                                 : fp8_wide_kernel<kGated, FI_DTYPE_F32>;
  };
  auto kern = gated ? pick(std::true_type{}) : pick(std::false_type{});
  static std::atomic<int> configured[kMaxDevices];
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= kMaxDevices) return set_cuda_error("cudaGetDevice");
  const int bit = 1 << (out * 2 + (gated ? 1 : 0));
  if (!(configured[dev] & bit)) {
    if (cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)kSmem) != cudaSuccess)
      return set_cuda_error("cudaFuncSetAttribute(fp8 wide smem)");
    configured[dev] |= bit;
  }
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = 2;
  attr[1].val.clusterDim.y = 1;
  attr[1].val.clusterDim.z = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)(2 * std::min<int64_t>(w.tiles, device_sm_count() / 2)));
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = kSmem;
  cfg.stream = stream;
  cfg.attrs = attr;
  cfg.numAttrs = 2;
  if (cudaLaunchKernelEx(&cfg, kern, w, ta, tw[0], tw[1]) != cudaSuccess) return set_cuda_error("fp8_wide_kernel launch");
  return FI_OK;
}

}  // namespace fi
