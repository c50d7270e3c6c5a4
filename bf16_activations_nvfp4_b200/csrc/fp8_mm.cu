// 8-bit products with a scale per block of 128 (sm_100a: tcgen05 + TMA + TMEM).
//
//   out[i][j] = sum_b As[i][b] * Ws[j / 128][b] * (sum over the 128 k of block b of A[i][k] W[j][k])
//
// and its gated form, silu(g) * u with g and u two such products of the same activations.
//
// The scales change every 128 k, so the tensor core sums one block of k at a time into a fresh
// TMEM buffer and the epilogue warps add it, times the block's scale, to fp32 accumulators in
// registers while the tensor core works on the next block.
//
// Here the weights are the MMA's M side (128 rows) and up to 256 activation rows its N side, so
// a weight byte is read once per 256 rows and one row costs no more than 16. Roles of a CTA:
//   warp 0    TMA producer: 128 x 128 weight tiles (two for the gated form) and N x 128
//             activation tiles into a ring, 128-byte swizzled;
//   warp 1    one thread issues the MMAs (four K = 32 steps per block) and the commits;
//   warp 2    the scales: As * Ws of four blocks at a time, up to eight blocks ahead, into a ring;
//   warps 3.. epilogue, one thread per weight row (two groups of four warps halve the columns,
//             or take the gate and the up tile): packed FMAs, two columns each.
// K splits are the CTAs of one cluster: their fp32 sums meet in distributed shared memory, where
// each CTA adds a slice of the outputs in split order. No workspace, no atomics, one launch.
//
// Bound by HBM up to some 128 rows: one row of 4096 x 14336 takes 12.2 us (4.8 TB/s; 3 to 4 us are
// the pipeline's start and the cluster's end), of 248320 x 5120 184 us (6.9 TB/s), the gated form
// at 16 rows of 2 x 17408 x 5120 30 us (6.0 TB/s). Up to 64 rows, and up to 96 where there are
// tiles enough, two CTAs share an SM, so that one's loads cover the other's start and end; above, a
// CTA has the SM's tensor memory to itself. 128 rows of 4096 x 14336 take 17.9 us, 256 rows 28.8.
//
// Every wait is bounded. On a timeout the roles stop, the producer and the MMA issuer wait,
// bounded, for what they have in flight, and every thread still meets the barriers. Every role waits for the
// end of the preceding kernel before its first bounded wait, so that a limit never counts another
// kernel's time.
#include <cstdint>
#include <algorithm>
#include <atomic>

#include <cuda.h>

#include "fp8_tc.cuh"

namespace fi {

namespace {

constexpr int kTileRows = 128;                     // weight rows per tile (the MMA's M)
constexpr uint32_t kTileBytes = kTileRows * 128;   // a tile of one k block
constexpr int kGroup = 4, kGroups = 2;             // blocks of k whose scales share a barrier; groups in the ring
constexpr int kWarpTma = 0, kWarpMma = 1, kWarpScale = 2, kWarpEpi0 = 3;
constexpr int kMaxStages = 10, kMaxBufs = 4;
constexpr int kMaxSplits = kFp8MaxSplits;

// The geometry of one instance: N activation rows per tile, one weight tile or two (gated).
template <int N, bool GATED>
struct Geo {
  static constexpr int kTiles = GATED ? 2 : 1;
  static constexpr int kEpiWarps = GATED || N > 64 ? 8 : 4;
  static constexpr int kThreads = (kWarpEpi0 + kEpiWarps) * 32;
  static constexpr int kCols = !GATED && N > 64 ? N / 2 : N;  // accumulators per epilogue thread
  static constexpr uint32_t kStageBytes = kTiles * kTileBytes + N * 128;
  static constexpr int kCtas = (GATED ? N <= 32 : N <= 96) ? 2 : 1;  // resident per SM
  static constexpr int kTmemCols = 512 / kCtas < kTiles * N * 4 ? 512 / kCtas : kTiles * N * 4;
  static constexpr uint32_t kBudget = kCtas == 2 ? 112 * 1024 : 226 * 1024;
  static constexpr uint32_t kScaleBytes = kGroups * kGroup * kTiles * N * 4;
  static constexpr uint32_t kFixed = 1024 + kScaleBytes + (2 * kMaxStages + kMaxBufs + 2 * kGroups + 1) * 8 + 64;
  static constexpr int kStages =
      (kBudget - kFixed) / kStageBytes < kMaxStages ? (kBudget - kFixed) / kStageBytes : kMaxStages;
  // Blocks the tensor core may be ahead of the epilogue: not more than there are stages, since a
  // stage's barrier tells the epilogue of its block, too, by one bit of its phase; twice on, it would read as not
  // there yet.
  static constexpr int kTmemBufs = kTmemCols / (kTiles * N);
  static constexpr int kBufs = kTmemBufs < kStages ? kTmemBufs : kStages;
  static constexpr uint32_t kRing = kStages * kStageBytes;
  static constexpr uint32_t kSmem = kFixed + kRing;
  static_assert(kStages >= 3, "ring");
  static_assert(kBufs >= 2 && kBufs <= kStages && kBufs <= kMaxBufs && kBufs * kTiles * N <= kTmemCols, "TMEM");
  static_assert((uint32_t)(kTiles * N) * kTileRows * 4 <= kRing, "the split sums reuse the ring");
};

template <int N, bool GATED>
__global__ void __launch_bounds__(Geo<N, GATED>::kThreads, Geo<N, GATED>::kCtas)
    fp8_mm_kernel(const Fp8MmArgs p, const __grid_constant__ CUtensorMap tmap_a,
                  const __grid_constant__ CUtensorMap tmap_w0, const __grid_constant__ CUtensorMap tmap_w1) {
  using G = Geo<N, GATED>;
  extern __shared__ __align__(1024) uint8_t smem_raw[];
  __shared__ volatile int abort_flag;
  __shared__ uint32_t tmem_slot;
  const uint32_t raw_s = smem_addr(smem_raw);
  const uint32_t base = (raw_s + 1023u) & ~1023u;
  uint8_t* const basep = smem_raw + (base - raw_s);
  float* const scales = reinterpret_cast<float*>(basep + G::kRing);  // [group][block][tile][N]
  uint64_t* const full = reinterpret_cast<uint64_t*>(basep + G::kRing + G::kScaleBytes);
  uint64_t* const done = full + G::kStages;  // a block's MMAs are complete: its stage may be refilled, its sums read
  uint64_t* const tmem_empty = done + G::kStages;
  uint64_t* const scale_full = tmem_empty + G::kBufs;
  uint64_t* const scale_empty = scale_full + kGroups;
  uint64_t* const drain = scale_empty + kGroups;

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int S = p.splits;
  const int split = (int)(blockIdx.x % (unsigned)S);
  const int64_t unit = blockIdx.x / (unsigned)S;
  const int64_t tile_n = unit / p.tiles_m;
  const int64_t m0 = (unit - tile_n * p.tiles_m) * N;
  const int kb0 = (int)((int64_t)split * p.kblocks / S);
  const int KB = (int)((int64_t)(split + 1) * p.kblocks / S) - kb0;
  const int rows = (int)min((int64_t)N, p.m - m0);  // activation rows of this tile

  if (threadIdx.x == 0) {
    abort_flag = 0;
    for (int i = 0; i < G::kStages; ++i) {
      mbar_init(&full[i], 1);
      mbar_init(&done[i], 1);
    }
    for (int i = 0; i < G::kBufs; ++i) {
      mbar_init(&tmem_empty[i], G::kEpiWarps);
    }
    for (int i = 0; i < kGroups; ++i) {
      mbar_init(&scale_full[i], 1);
      mbar_init(&scale_empty[i], G::kEpiWarps);
    }
    mbar_init(drain, 1);
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
  }
  if (warp == kWarpMma) {
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_addr(&tmem_slot)),
                 "r"((uint32_t)G::kTmemCols)
                 : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
  }
  asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory");
  __syncthreads();
  asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
  const uint32_t tmem = tmem_slot;
  // waited for before the first access to another CTA's shared memory: they have all started
  asm volatile("barrier.cluster.arrive.relaxed.aligned;" ::: "memory");
  pdl_launch_dependents();

  if (warp == kWarpTma) {
    if (lane == 0) {
      prefetch_map(&tmap_w0);
      if (GATED) prefetch_map(&tmap_w1);
      prefetch_map(&tmap_a);
      // while the kernel before this one ends: the first weights on their way to L2
      for (int i = 0; i < KB && i < G::kStages; ++i) {
        tma_prefetch_2d(&tmap_w0, (kb0 + i) * kFp8Block, (int)(tile_n * kTileRows));
        if (GATED) tma_prefetch_2d(&tmap_w1, (kb0 + i) * kFp8Block, (int)(tile_n * kTileRows));
      }
      const uint64_t once = evict_first_policy();
      pdl_wait();
      int issued = 0;
      for (int i = 0; i < KB && !p.debug_stall; ++i) {
        const int st = i % G::kStages;
        if (i >= G::kStages &&
            !mbar_wait_spin(&done[st], ((i / G::kStages) - 1) & 1, &abort_flag, p.timeout_ns, p.err, 2u))
          break;
        const uint32_t dst = base + (uint32_t)st * G::kStageBytes;
        const int x = (kb0 + i) * kFp8Block;
        mbar_arrive_expect_tx(&full[st], G::kStageBytes);
        tma_load_2d_hint(dst, &tmap_w0, x, (int)(tile_n * kTileRows), smem_addr(&full[st]), once);
        if (GATED)
          tma_load_2d_hint(dst + kTileBytes, &tmap_w1, x, (int)(tile_n * kTileRows), smem_addr(&full[st]), once);
        tma_load_2d(dst + G::kTiles * kTileBytes, &tmap_a, x, (int)m0, smem_addr(&full[st]));
        issued = i + 1;
      }
      // the copies in flight land before the CTA's shared memory is given up
      volatile int never = 0;
      for (int i = max(0, issued - G::kStages); i < issued; ++i)
        mbar_wait_spin(&full[i % G::kStages], (i / G::kStages) & 1, &never, p.timeout_ns, p.err, 4u);
    }
    __syncwarp();
  } else if (warp == kWarpMma) {
    if (lane == 0) {
      constexpr uint32_t idesc = f8_idesc(kTileRows, N);
      bool ok = true;
      pdl_wait();  // the limit of a wait counts from the preceding kernel's end
      for (int i = 0; i < KB; ++i) {
        const int st = i % G::kStages, b = i % G::kBufs;
        ok = mbar_wait_spin(&full[st], (i / G::kStages) & 1, &abort_flag, p.timeout_ns, p.err, 1u) &&
             (i < G::kBufs ||
              mbar_wait_spin(&tmem_empty[b], ((i / G::kBufs) - 1) & 1, &abort_flag, p.timeout_ns, p.err, 1u));
        if (!ok) break;
        asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
        const uint32_t stage = base + (uint32_t)st * G::kStageBytes;
        const uint64_t bdesc = sw128_desc(stage + G::kTiles * kTileBytes);
#pragma unroll
        for (int t = 0; t < G::kTiles; ++t) {
          const uint64_t adesc = sw128_desc(stage + t * kTileBytes);
          const uint32_t d = tmem + (uint32_t)((b * G::kTiles + t) * N);
#pragma unroll
          for (int s = 0; s < 4; ++s)  // K = 32 bytes each
            umma_f8(d, adesc + (uint64_t)(2 * s), bdesc + (uint64_t)(2 * s), idesc, s > 0);
        }
        umma_commit(&done[st]);
      }
      if (!ok) {  // the MMAs in flight end before TMEM is freed
        volatile int never = 0;
        umma_commit(drain);
        mbar_wait_spin(drain, 0, &never, p.timeout_ns, p.err, 8u);
      }
    }
    __syncwarp();
  } else if (warp == kWarpScale) {
    pdl_wait();
    constexpr int kPer = (N + 31) / 32, kAhead = 4;
    float sa[kAhead][kPer], sw[kAhead][G::kTiles];
    auto load = [&](int i, int d) {
#pragma unroll
      for (int r = 0; r < kPer; ++r) {
        const int row = lane + 32 * r;
        sa[d][r] = i < KB && row < rows ? __ldg(p.As + (m0 + row) * p.kblocks + kb0 + i) : 0.0f;
      }
#pragma unroll
      for (int t = 0; t < G::kTiles; ++t)
        sw[d][t] = i < KB ? __ldg(p.Ws[t] + tile_n * p.kblocks + kb0 + i) : 0.0f;
    };
#pragma unroll
    for (int d = 0; d < kAhead; ++d) load(d, d);
    static_assert(kAhead == kGroup, "a group is one batch of loads");
    bool ok = true;
    for (int i0 = 0; i0 < KB && ok; i0 += kGroup) {
      const int g = i0 / kGroup % kGroups;
      if (i0 >= kGroups * kGroup)
        ok = mbar_wait_spin(&scale_empty[g], (i0 / (kGroup * kGroups) - 1) & 1, &abort_flag, p.timeout_ns, p.err, 2u);
      ok = __all_sync(0xffffffffu, ok);
      if (!ok) break;
      float* dst = scales + g * (kGroup * G::kTiles * N);
#pragma unroll
      for (int d = 0; d < kGroup; ++d) {
#pragma unroll
        for (int t = 0; t < G::kTiles; ++t)
#pragma unroll
          for (int r = 0; r < kPer; ++r)
            if (lane + 32 * r < N) dst[(d * G::kTiles + t) * N + lane + 32 * r] = sa[d][r] * sw[d][t];
        load(i0 + kGroup + d, d);
      }
      __syncwarp();
      if (lane == 0) mbar_arrive(&scale_full[g]);
    }
  } else {
    pdl_wait();  // before the first wait with a limit, and before any output is written
    const int epi = warp - kWarpEpi0, quarter = warp & 3, group = epi >> 2;
    const int tile = GATED ? group : 0;
    const int c0 = GATED ? 0 : group * G::kCols;  // first activation row (column) of this thread
    const int wrow = quarter * 32 + lane;         // weight row in the tile
    float acc[G::kCols];
#pragma unroll
    for (int c = 0; c < G::kCols; ++c) acc[c] = 0.0f;
    // A wait that runs out raises the abort flag; the ones after it then give up at once, and the
    // blocks' sums are what TMEM held. The flag is looked at now and then.
    const uint32_t done0 = smem_addr(done), done_end = done0 + G::kStages * 8;
    const uint32_t sp0 = smem_addr(scales) + (uint32_t)(tile * N + c0) * 4;
    uint32_t done_bar = done0, phase = 0;
#pragma unroll 1
    for (int i = 0; i < KB; ++i) {
      const int b = i % G::kBufs;
      if (i % 64 == 63 && __any_sync(0xffffffffu, abort_flag != 0)) break;
      if (i % kGroup == 0)
        mbar_wait_spin(&scale_full[i / kGroup % kGroups], i / (kGroup * kGroups) & 1, &abort_flag, p.timeout_ns, p.err,
                       16u);
      mbar_wait_addr(done_bar, phase, &abort_flag, p.timeout_ns, p.err, 16u);
      __syncwarp();
      asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
      done_bar += 8;
      if (done_bar == done_end) {
        done_bar = done0;
        phase ^= 1;
      }
      const uint32_t taddr = tmem + ((uint32_t)(quarter * 32) << 16) + (uint32_t)((b * G::kTiles + tile) * N + c0);
      const uint32_t sp = sp0 + (uint32_t)(i % (kGroup * kGroups)) * (G::kTiles * N * 4);
      // columns in flight from TMEM: all of them where the registers allow it
      constexpr int kChunk = G::kCols == 64 ? (G::kCtas == 1 ? 64 : 32) : (G::kCols == 32 ? 32 : 16);
#pragma unroll
      for (int c = 0; c < G::kCols; c += kChunk) {
        uint32_t d[kChunk];
        tmem_ld_async(taddr + c, d);
        tmem_wait_ld(d);
        if (c + kChunk == G::kCols) {
          // everything is in registers: the buffer is free
          asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory");
          __syncwarp();
          if (lane == 0) mbar_arrive(&tmem_empty[b]);
        }
#pragma unroll
        for (int q = 0; q < kChunk; q += 4) {
          uint64_t s01, s23;
          asm volatile("ld.shared.v2.u64 {%0, %1}, [%2];" : "=l"(s01), "=l"(s23) : "r"(sp + (uint32_t)(c + q) * 4));
          fma_scaled(acc[c + q], acc[c + q + 1], d[q], d[q + 1], s01);
          fma_scaled(acc[c + q + 2], acc[c + q + 3], d[q + 2], d[q + 3], s23);
        }
      }
      if (i % kGroup == kGroup - 1) {
        __syncwarp();
        if (lane == 0) mbar_arrive(&scale_empty[i / kGroup % kGroups]);
      }
    }
    // the ring is free: every copy has landed and every MMA has read its operands
    float* part = reinterpret_cast<float*>(basep) + (tile * N + c0) * kTileRows + wrow;
#pragma unroll
    for (int c = 0; c < G::kCols; ++c)
      if (c0 + c < rows) part[c * kTileRows] = acc[c];
  }

  asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory");
  __syncwarp();
  // Where a wait of any CTA of the cluster ran out, the sums are not the blocks': nothing is stored. The CTA
  // that gave up tells the others. (Read from them by each warp, the flags took 0.25 us of the 9.8 of
  // 64 x 5120 x 5120; a mark in the sums took as much.)
  asm volatile("barrier.cluster.wait.aligned;" ::: "memory");
  if (abort_flag)
    for (int r = 0; r < S; ++r) st_dsmem_u32(const_cast<int*>(&abort_flag), (uint32_t)r, 1);
  __syncwarp();
  cluster_sync();
  const bool sound = abort_flag == 0;
  // four outputs of one activation row at a time: all splits' sums are on their way before the
  // first is added
  const int quads = rows * (kTileRows / 4);
  const int chunk = (quads + S - 1) / S;
  const int q_end = min(quads, (split + 1) * chunk);
  const bool wide = p.n % 4 == 0 && (reinterpret_cast<uintptr_t>(p.out) & 15) == 0;
  for (int e = split * chunk + (int)threadIdx.x; e < q_end; e += G::kThreads) {
    const int64_t j = tile_n * kTileRows + (e & (kTileRows / 4 - 1)) * 4;
    float4 v[G::kTiles];
#pragma unroll
    for (int t = 0; t < G::kTiles; ++t) {
      const uint32_t at = base + (uint32_t)(t * N * kTileRows + e * 4) * 4u;
      float4 part[kMaxSplits];
#pragma unroll
      for (int r = 0; r < kMaxSplits; ++r)
        if (r < S) part[r] = ld_dsmem_v4(at, (uint32_t)r);
      v[t] = part[0];
#pragma unroll
      for (int r = 1; r < kMaxSplits; ++r) {
        if (r < S) {
          v[t].x = __fadd_rn(v[t].x, part[r].x);
          v[t].y = __fadd_rn(v[t].y, part[r].y);
          v[t].z = __fadd_rn(v[t].z, part[r].z);
          v[t].w = __fadd_rn(v[t].w, part[r].w);
        }
      }
    }
    if (GATED) {
      const float4 u = v[G::kTiles - 1];
      silu_times(v[0].x, v[0].y, u.x, u.y);
      silu_times(v[0].z, v[0].w, u.z, u.w);
    }
    if (sound && j < p.n)
      store_out4(p.out, p.out_dtype, (m0 + e / (kTileRows / 4)) * p.n + j, v[0], wide, p.n - j);
  }
  __syncwarp();
  cluster_sync();  // no CTA leaves while another reads its sums
  if (warp == kWarpMma) {
    asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"((uint32_t)G::kTmemCols)
                 : "memory");
  }
}

// ---------------------------------------------------------------------------- host side

// Launched never: stands for the kernels' shape in the occupancy query.
__global__ void shape_kernel() {}

// How a call is cut, and what it is expected to take, in tenths of a block of the CTA-pair kernel (a
// block of 128 k of one tile there takes about 0.36 us).
struct Cut {
  int splits;
  int64_t units;  // tiles of weight rows x tiles of activation rows
  int64_t cost;
};

// What a tile of N activation rows takes, as measured on B200 (a tenth of a block of the CTA-pair kernel is
// 36 ns): a block of k; a wave's start and end; for each row that a CTA writes, in tenths. A wave of a
// tile that competes with no other counts 7 us, its writing included.
struct TileCost {
  int block, wave, row;
};
template <int N, bool GATED>
constexpr TileCost tile_cost() {
  if constexpr (GATED) {
    if (N == 128) return {24, 145, 8};  // 0.9 us a block, 5.2 us a wave, 0.03 us a row
    if (N == 64) return {11, 185, 8};   // 0.4, 6.7
  } else {
    if (N == 256) return {20, 145, 8};  // 0.72, 5.2
    if (N == 128) return {10, 145, 8};  // 0.37, 5.2
    if (N == 96) return {18, 200, 0};   // 0.65 with two CTAs on every SM
  }
  return {9, 200, 0};
}

// The split of least cost, or the given one: waves of clusters, each with its blocks of k, a start and
// an end, and the meeting of a cluster (1.4 us). The gated N = 128, whose splits have twice as much
// to read from one another, writes half of its rows' cost whatever the split, and 0.2 us a split.
template <int N, bool GATED>
int cut_tiles(const Fp8MmArgs& a, int splits, Cut* out) {
  using G = Geo<N, GATED>;
  const int sms = device_sm_count();
  auto kern = fp8_mm_kernel<N, GATED>;
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= kMaxDevices) return set_cuda_error("cudaGetDevice");
  static std::atomic<int> active[kMaxDevices][kMaxSplits + 1];  // clusters of s CTAs the device holds at once; [0]: set up
  if (!active[dev][0]) {
    if (cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)G::kSmem) != cudaSuccess ||
        cudaFuncSetAttribute(shape_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmemBudget + 1024) !=
            cudaSuccess)
      return set_cuda_error("cudaFuncSetAttribute(fp8 smem)");
    // The query answers one CTA per SM for a kernel that allocates TMEM, where the device holds as
    // many as TMEM and shared memory allow: asked for a kernel of the same shape without TMEM.
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.y = 1;
    attr[0].val.clusterDim.z = 1;
    cudaLaunchConfig_t cfg = {};
    cfg.blockDim = dim3(G::kThreads);
    cfg.dynamicSmemBytes = G::kSmem + 1024;  // with the kernel's static shared memory
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    for (int s = 1; s <= kMaxSplits; ++s) {
      // a cluster lies within one GPU processing cluster, so fewer fit than SMs / s
      int n = 0;
      attr[0].val.clusterDim.x = (unsigned)s;
      cfg.gridDim = dim3((unsigned)(s * sms));
      if (cudaOccupancyMaxActiveClusters(&n, shape_kernel, &cfg) != cudaSuccess || n < 1) {
        (void)cudaGetLastError();
        n = std::max(1, sms * G::kCtas / s);
      }
      active[dev][s] = n;
    }
    active[dev][0] = 1;
  }
  constexpr TileCost kCost = tile_cost<N, GATED>();
  constexpr bool kTwice = GATED && N == 128;
  const int64_t rows = std::min<int64_t>(a.m, N) * kCost.row / 10;
  out->units = (a.n + kTileRows - 1) / kTileRows * ((a.m + N - 1) / N);
  out->cost = -1;
  const int most = std::min(splits == 0 ? kMaxSplits : splits, a.kblocks);
  for (int s = splits == 0 ? 1 : most; s <= most; ++s) {
    const int64_t at_once = active[dev][s];
    const int64_t write = s > 1 && kTwice ? rows / 2 + 6 * s : rows / s;
    const int64_t wave = (a.kblocks + s - 1) / s * kCost.block + kCost.wave + write;
    const int64_t cost = (out->units + at_once - 1) / at_once * wave + (s > 1 ? 40 : 0);
    if (out->cost < 0 || cost < out->cost) {
      out->cost = cost;
      out->splits = s;
    }
  }
  return FI_OK;
}

template <int N, bool GATED>
int launch_tile(Fp8MmArgs a, const Cut& cut, cudaStream_t stream) {
  using G = Geo<N, GATED>;
  a.tiles_m = (int)((a.m + N - 1) / N);
  a.splits = cut.splits;
  const int64_t units = cut.units;
  const int64_t grid = units * a.splits;
  if (grid > 0x7fffffffLL || a.n > 0x7fffff00LL || a.m > 0x7fffff00LL || a.k > 0x7fffff00LL)
    return set_error(FI_ERR_UNSUPPORTED_SHAPE, "m=%lld n=%lld k=%lld is too large", (long long)a.m, (long long)a.n,
                     (long long)a.k);
  CUtensorMap ta, tw[2];
  int rc = encode_codes(&ta, a.A, a.k, a.m, N);
  for (int t = 0; t < G::kTiles && rc == FI_OK; ++t) rc = encode_codes(&tw[t], a.W[t], a.k, a.n, kTileRows);
  if (rc != FI_OK) return rc;
  if (!GATED) tw[1] = tw[0];
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = (unsigned)a.splits;
  attr[0].val.clusterDim.y = 1;
  attr[0].val.clusterDim.z = 1;
  attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[1].val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)grid);
  cfg.blockDim = dim3(G::kThreads);
  cfg.dynamicSmemBytes = G::kSmem;
  cfg.stream = stream;
  cfg.attrs = attr;
  cfg.numAttrs = 2;
  if (cudaLaunchKernelEx(&cfg, fp8_mm_kernel<N, GATED>, a, ta, tw[0], tw[1]) != cudaSuccess)
    return set_cuda_error("fp8_mm_kernel launch");
  return FI_OK;
}

// What the CTA-pair kernel is expected to take: 0.36 us a block (0.4 where one row of tiles reads
// all weights and HBM counts), 4 us a wave and 2.5 us a call.
int64_t wide_cost(const Fp8MmArgs& a, bool gated) {
  const int64_t tiles_m = (a.m + 255) / 256, tiles = tiles_m * ((a.n + (gated ? 127 : 255)) / (gated ? 128 : 256));
  const int64_t pairs = std::max(1, device_sm_count() / 2);
  return (tiles + pairs - 1) / pairs * (a.kblocks * (gated && tiles_m == 1 ? 11 : 10) + 110) + 70;
}

// The cheapest of two tiles of this kernel and, where `pair` says so, the CTA-pair kernel. Measured
// (us):
//   65 to 96 rows, tiles of 96 rows two to an SM / of 128 one to an SM: 77 of 10304 x 2688 11.7 / 13.9,
//   80 of 34816 x 5120 37.3 / 43.3, 96 of 248320 x 5120 280 / 315, of 4096 x 4096 12.0 / 9.7;
//   from 129 rows on, tiles of 128 / 256 / CTA pairs: 256 of 178 x 768 5.6 / 8.1 / 8.3, of 2048 x 7168
//   12.0 / 15.4 / 25.6, 130 of 4096 x 14336 28.1 / 25.3 / 46.6, 391 of 4096 x 4096 20.9 / 20.5 / 17.7,
//   256 of 5295 x 416 10.1 / 16.0 / 8.5, 1000 of 4096 x 4096 41.4 / 35.0 / 18.9;
//   gated from 65 rows on, tiles of 64 / 128 / CTA pairs: 128 of 65 x 11408 11.5 / 18.1 / 38.3, of
//   1746 x 1136 8.6 / 10.7 / 9.2, of 17408 x 5120 53.9 / 44.5 / 45.5, 200 of 8192 x 2048 30.3 / 24.6 / 13.2.
template <int N1, int N2, bool GATED>
int launch_cheapest(const Fp8MmArgs& a, int splits, bool pair, cudaStream_t stream) {
  Cut one, two;
  int rc = cut_tiles<N1, GATED>(a, splits, &one);
  if (rc == FI_OK) rc = cut_tiles<N2, GATED>(a, splits, &two);
  if (rc != FI_OK) return rc;
  if (pair && wide_cost(a, GATED) < std::min(one.cost, two.cost)) return launch_fp8_wide(a, GATED, stream);
  return one.cost < two.cost ? launch_tile<N1, GATED>(a, one, stream) : launch_tile<N2, GATED>(a, two, stream);
}

template <int N, bool GATED>
int launch_only(const Fp8MmArgs& a, int splits, cudaStream_t stream) {
  Cut cut;
  const int rc = cut_tiles<N, GATED>(a, splits, &cut);
  return rc != FI_OK ? rc : launch_tile<N, GATED>(a, cut, stream);
}

}  // namespace

int launch_fp8_mm(Fp8MmArgs a, bool gated, int splits, cudaStream_t stream) {
  a.err = device_error_word();
  if (!a.err) return set_cuda_error("cudaGetSymbolAddress(device error word)");
  a.timeout_ns = wait_timeout_ns();
  a.debug_stall = take_debug_stall();
  const bool pair = splits <= 1;  // the CTA-pair kernel has no splits
  if (gated) {
    if (a.m <= 16) return launch_only<16, true>(a, splits, stream);
    if (a.m <= 32) return launch_only<32, true>(a, splits, stream);
    if (a.m <= 64) return launch_only<64, true>(a, splits, stream);
    return launch_cheapest<64, 128, true>(a, splits, pair, stream);
  }
  if (a.m <= 16) return launch_only<16, false>(a, splits, stream);
  if (a.m <= 32) return launch_only<32, false>(a, splits, stream);
  if (a.m <= 64) return launch_only<64, false>(a, splits, stream);
  if (a.m <= 96) return launch_cheapest<96, 128, false>(a, splits, false, stream);
  return launch_cheapest<128, 256, false>(a, splits, pair && a.m > 128, stream);
}

}  // namespace fi
