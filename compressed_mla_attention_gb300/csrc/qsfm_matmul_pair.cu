// Products of e4m3 rows with e4m3 matrices where a group has many rows (sm_103a); the
// formula and the kernel of few rows are in qsfm_matmul.cu.
//
// Two CTAs of a pair share a tile of 256 rows of a by 256 matrix rows (tcgen05.mma
// cta_group::2): each loads its own 128 rows of a and half of the matrix's, 32 KB a block
// of K. Rows of a are the tensor-memory lanes: a thread's 128 sums are those of one row
// with 128 matrix rows, which have one scale, so a block's factor is one number a thread.
//
// Per CTA: a warp that loads, two that issue MMAs (of the pair's first CTA alone), one
// that copies scales, eight that add up and store. A block's MMAs take 512 cycles;
// meanwhile the eight warps read the previous one's 128 x 256 products out of tensor
// memory and add them up. What it took (cycles a block, K = 8192):
//  * a release of an accumulator at the cluster's scope waits for all the thread's memory
//    operations: 2800 -> 1250 without;
//  * single FMAs instead of pairs (fma.rn.f32x2: 64 a thread took longer than 128): 960;
//  * scales through shared memory, eight blocks at a time, instead of 4-byte loads: 770.
// At 770 the GPU is at its power limit (1660 MHz of 2070 in a loop): 8192 x 8192 x 8192 in
// 385 us (2.86 PFLOP/s), 420 in a loop; a library's product of the same codes without
// scales 330 in a loop. Tried: tiles of 192 matrix rows (one round of loads from tensor
// memory, an earlier release) 460; two MMAs of 128 matrix rows each 500, before the last
// step.
#include <atomic>

#include "qsfm_matmul_common.cuh"

namespace qsfm {
namespace {

constexpr int kPairRows = 256;    // rows of a of a tile: 128 a CTA
constexpr int kPairCols = 256;    // matrix rows of a tile: each CTA holds half of them
constexpr int kSums = kPairCols / 2;  // of an adding thread
constexpr int kRound = 64;             // products of a thread on their way from tensor memory
constexpr int kPairBlock = 8;     // row tiles that are walked before the next of the matrix's
constexpr int kAddWarps = 8;
constexpr int kPairThreads = 32 * (kAddWarps + 4);
constexpr int kAddRegs = 224, kOtherRegs = 56, kLaunchRegs = 168;
static_assert(256 * kAddRegs + 128 * kOtherRegs <= kPairThreads * kLaunchRegs, "registers");
constexpr uint32_t kARows = 128 * kMmK;                       // a CTA's rows of a
constexpr uint32_t kPairStage = kARows + kPairCols / 2 * kMmK;  // and of the matrix
constexpr int kPairStages = 6;
constexpr uint32_t kOutWarp = 2048;  // 32 rows x 64 bytes
constexpr uint32_t kOutAt = kPairStages * kPairStage;  // of each adding warp: sums on their way out
constexpr int kPairSlots = 3, kSlotBlocks = 8;  // scales of 8 blocks of K at a time
constexpr uint32_t kSlotBlock = 512 + 16;       // 128 rows' scales, one of the matrix's for each half
constexpr uint32_t kScaleAt = kOutAt + kAddWarps * kOutWarp;
constexpr uint32_t kPrefixAt = kScaleAt + kPairSlots * kSlotBlocks * kSlotBlock;
constexpr uint32_t kBarAt = (kPrefixAt + (kMmMaxGroups + 4) * 4 + 7) & ~7u;
constexpr uint32_t kPairSmem = kBarAt + 256 + 1024;
static_assert(kPairSmem <= kMmSmemMax, "shared memory");
constexpr uint32_t kPairTmem = 512, kAccAt = 256;  // two accumulators, 256 columns apart

// barriers; those marked * are used in the first CTA alone
constexpr int kPbFull = 0 /* * both CTAs' copies */, kPbEmpty = kPairStages, kPbTFull = 2 * kPairStages,
              kPbTEmpty = kPbTFull + 2 /* * both CTAs' adding warps */, kPbDrain = kPbTEmpty + 2 /* * of each issuing warp */,
              kPbSFull = kPbDrain + 2, kPbSEmpty = kPbSFull + kPairSlots, kPbCount = kPbSEmpty + kPairSlots;
static_assert(kPbCount * 8 + 8 <= 256, "barriers");

struct PairShape {
  int kb;         // blocks of K
  int col_tiles;  // tiles of the matrix's rows
  int col_blocks; // scales along the matrix's rows
};

// A copy into this CTA's shared memory that completes on a barrier of the pair's first CTA.
__device__ __forceinline__ void pair_load_2d(uint32_t dst, const void* tmap, int x, int y, uint32_t bar) {
  asm volatile(
      "cp.async.bulk.tensor.2d.cta_group::2.shared::cluster.global.mbarrier::complete_tx::bytes"
      " [%0], [%1, {%2, %3}], [%4];" ::"r"(dst),
      "l"(reinterpret_cast<uint64_t>(tmap)), "r"(x), "r"(y), "r"(bar)
      : "memory");
}
__device__ __forceinline__ void pair_load_3d(uint32_t dst, const void* tmap, int x, int y, int z, uint32_t bar) {
  asm volatile(
      "cp.async.bulk.tensor.3d.cta_group::2.shared::cluster.global.mbarrier::complete_tx::bytes"
      " [%0], [%1, {%2, %3, %4}], [%5];" ::"r"(dst),
      "l"(reinterpret_cast<uint64_t>(tmap)), "r"(x), "r"(y), "r"(z), "r"(bar)
      : "memory");
}
// Arrives on `bar` of both CTAs once the pair's MMAs issued so far have completed.
__device__ __forceinline__ void pair_commit(uint64_t* bar) {
  asm volatile(
      "{\n .reg .pred e;\n .reg .b16 both;\n mov.b16 both, 3;\n elect.sync _|e, 0xffffffff;\n"
      " @e tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64 [%0], both;\n}"
      ::"r"(smem_u32(bar))
      : "memory");
}
// (What it orders is tensor memory's reads, by tcgen05.fence; a release at the cluster's
// scope would wait for every load and store of the thread before it.)
__device__ __forceinline__ void arrive_in_cluster(uint32_t bar) {
  asm volatile("mbarrier.arrive.shared::cluster.b64 _, [%0];" ::"r"(bar) : "memory");
}

// The pair's walk over the tiles.
struct PairWalk {
  const int* prefix;
  int g, at, step, total;
  __device__ __forceinline__ bool next(const qsfm_matmul_params& p, const PairShape& s, MmTile& t) {
    if (at >= total) return false;
    while (at >= prefix[g + 1]) ++g;
    int lo, hi;
    bool bad;
    group_rows(p, g, lo, hi, bad);
    const int row_tiles = (hi - lo + kPairRows - 1) / kPairRows;
    const int local = at - prefix[g], block = local / (kPairBlock * s.col_tiles);
    const int rest = local - block * (kPairBlock * s.col_tiles), high = min(kPairBlock, row_tiles - block * kPairBlock);
    const int n = rest / high, m = block * kPairBlock + rest - n * high;
    t.g = g;
    t.n0 = n * kPairCols;
    t.row0 = lo + m * kPairRows;
    t.cols = min(kPairRows, hi - t.row0);  // rows of the tile
    at += step;
    return true;
  }
};

__device__ void pair_load(const qsfm_matmul_params& p, const PairShape& s, const MmSmem& sm, PairWalk walk, uint32_t rank,
                          const CUtensorMap* amap, const CUtensorMap* wmap, int* fault) {
  if ((threadIdx.x & 31) != 0) return;
  uint32_t st = 0, par = 1;
  MmTile t;
  while (walk.next(p, s, t)) {
    for (int b = 0; b < s.kb; ++b) {
      if (!mm_wait(sm, kPbEmpty + st, par, fault)) return;
      const uint32_t at = sm.base + st * kPairStage, bar = in_cta(smem_u32(sm.bar(kPbFull + st)), 0);
      if (rank == 0) mbar_arrive_expect_tx(sm.bar(kPbFull + st), 2 * kPairStage);
      pair_load_2d(at, amap, b * kMmK, t.row0 + 128 * int(rank), bar);
      pair_load_3d(at + kARows, wmap, b * kMmK, t.n0 + kPairCols / 2 * int(rank), t.g, bar);
      if (++st == kPairStages) {
        st = 0;
        par ^= 1;
      }
    }
  }
}

// Two warps issue in turn, `odd` the second: waiting for a stage and an accumulator and
// handing four MMAs and two commits over takes one warp 550 cycles and more, longer than
// the MMAs themselves.
__device__ void pair_issue(const qsfm_matmul_params& p, const PairShape& s, const MmSmem& sm, PairWalk walk, uint32_t odd,
                           uint32_t tmem, int* fault) {
  // formats 0 (e4m3) for both operands, as in the bf16 descriptor's f16 form
  constexpr uint32_t idesc = make_idesc_bf16(kPairRows, kPairCols, 0, 0, true);
  static_assert(kPairStages % 2 == 0, "a warp's stages are every other one");
  const uint32_t d = tmem + odd * kAccAt;
  uint32_t st = odd, par = 0, tpar = 1, first = odd;  // first: whether the tile's first block is the other warp's
  MmTile t;
  while (walk.next(p, s, t)) {
    for (int b = int(first); b < s.kb; b += 2) {
      if (!mm_warp_wait2(sm, kPbFull + st, par, kPbTEmpty + odd, tpar, fault)) return;
      tc_fence_after();
      const uint32_t a = mm_desc(sm.base + st * kPairStage), w = a + (kARows >> 4);
      mma_e4m3<0, 2>(d, a, w, idesc, 0);
      mma_e4m3<2, 2>(d, a, w, idesc, 1);
      mma_e4m3<4, 2>(d, a, w, idesc, 1);
      mma_e4m3<6, 2>(d, a, w, idesc, 1);
      pair_commit(sm.bar(kPbTFull + odd));
      pair_commit(sm.bar(kPbEmpty + st));
      st += 2;
      if (st >= kPairStages) {
        st = odd;
        par ^= 1;
      }
      tpar ^= 1;
    }
    first ^= uint32_t(s.kb) & 1;
  }
}

// The warp's 32 rows of kSums sums (a lane has a row) to `out`, rows `stride` elements
// apart, of which the first `rows` and `cols` are there. 64 bytes of each row at a time go
// through shared memory (`stage`, 2 KB, a row's 16-byte pieces in turn by row), so that a
// warp stores whole sectors; single elements where the output is not aligned or ends.
template <typename T>
__device__ __forceinline__ void store_rows(T* out, size_t stride, const float (&acc)[kSums], int rows, int cols,
                                           bool aligned, uint8_t* stage) {
  constexpr int kPart = 64 / sizeof(T), kEach = 16 / sizeof(T);  // columns at a time, of a piece
  const int lane = threadIdx.x & 31;
  const auto at = [&](int r, int piece) { return stage + 64 * r + 16 * (piece ^ ((r >> 1) & 3)); };
#pragma unroll
  for (int c0 = 0; c0 < kSums; c0 += kPart) {
    if (c0 >= cols) break;
    __syncwarp();
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      uint32_t w[4];
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const int c = c0 + kEach * i + kEach / 4 * j;
        if constexpr (sizeof(T) == 4) {
          w[j] = __float_as_uint(acc[c]);
        } else if constexpr (__is_same(T, __half)) {
          w[j] = pack_f16(acc[c], acc[c + 1]);
        } else {
          const __nv_bfloat162 h = __floats2bfloat162_rn(acc[c], acc[c + 1]);
          w[j] = *reinterpret_cast<const uint32_t*>(&h);
        }
      }
      *reinterpret_cast<uint4*>(at(lane, i)) = make_uint4(w[0], w[1], w[2], w[3]);
    }
    __syncwarp();
    if (aligned && c0 + kPart <= cols) {
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int r = 8 * i + lane / 4, piece = lane % 4;
        const uint4 v = *reinterpret_cast<const uint4*>(at(r, piece));
        if (r < rows) *reinterpret_cast<uint4*>(out + r * stride + c0 + piece * kEach) = v;
      }
    } else {
      for (int i = lane; i < rows * kPart; i += 32) {
        const int r = i / kPart, c = i % kPart;
        if (c0 + c < cols) out[r * stride + c0 + c] = *reinterpret_cast<const T*>(at(r, c / kEach) + c % kEach * sizeof(T));
      }
    }
  }
}

// The scales of eight blocks at a time, on their way to shared memory with the loads: from
// global memory, a thread's own 4 bytes a block cost the adding warps a third of their time.
__device__ void pair_scales(const qsfm_matmul_params& p, const PairShape& s, const MmSmem& sm, PairWalk walk,
                            uint32_t rank, int* fault) {
  const int lane = threadIdx.x & 31;
  uint32_t slot = 0, par = 1;
  MmTile t;
  while (walk.next(p, s, t)) {
    // rows behind the tile's take its last one's scales, and are not stored
    const float* as[4];
#pragma unroll
    for (int i = 0; i < 4; ++i)
      as[i] = p.a_scale + size_t(t.row0 + min(128 * int(rank) + 32 * i + lane, t.cols - 1)) * p.a_scale_row_stride;
    // lane 0 and 1: of the two halves
    const float* ws = p.w_scale + (size_t(t.g) * s.col_blocks + min(t.n0 / 128 + (lane & 1), s.col_blocks - 1)) * s.kb;
    for (int b0 = 0; b0 < s.kb; b0 += kSlotBlocks) {
      if (!mm_warp_wait(sm, kPbSEmpty + slot, par, fault)) break;
      uint32_t at = sm.base + kScaleAt + slot * kSlotBlocks * kSlotBlock;
      for (int b = b0; b < min(b0 + kSlotBlocks, s.kb); ++b, at += kSlotBlock) {
#pragma unroll
        for (int i = 0; i < 4; ++i) cp_async4(at + 4 * (32 * i + lane), as[i] + size_t(b) * p.a_scale_col_stride, 4);
        if (lane < 2) cp_async4(at + 512 + 4 * lane, ws + b, 4);
      }
      cp_async_arrive(sm.bar(kPbSFull + slot));
      if (++slot == kPairSlots) {
        slot = 0;
        par ^= 1;
      }
    }
  }
  asm volatile("cp.async.wait_all;" ::: "memory");
}

__device__ void pair_sum(const qsfm_matmul_params& p, const PairShape& s, const MmSmem& sm, PairWalk walk, uint32_t rank,
                         uint32_t tmem, int* fault) {
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int row0 = 128 * int(rank) + 32 * (warp & 3), half = warp >> 2;
  const uint32_t tempty = in_cta(smem_u32(sm.bar(kPbTEmpty)), 0);
  const int size = p.out_type == QSFM_F32 ? 4 : 2;
  const bool aligned = (reinterpret_cast<uintptr_t>(p.out) & 15) == 0 && (p.out_row_stride * size) % 16 == 0;
  uint32_t buf = 0, tpar = 0, slot = 0, spar = 0;
  MmTile t;
  while (walk.next(p, s, t)) {
    float acc[kSums];
#pragma unroll
    for (int i = 0; i < kSums; ++i) acc[i] = 0.f;
    const int n0 = t.n0 + kSums * half;
    for (int b0 = 0; b0 < s.kb; b0 += kSlotBlocks) {
      if (!mm_warp_wait(sm, kPbSFull + slot, spar, fault)) return;
      const float* scales = reinterpret_cast<const float*>(sm.ptr + kScaleAt + slot * kSlotBlocks * kSlotBlock);
      for (int b = b0; b < min(b0 + kSlotBlocks, s.kb); ++b, scales += kSlotBlock / 4) {
        const float f = scales[32 * (warp & 3) + lane] * scales[128 + half];
        if (!mm_warp_wait(sm, kPbTFull + buf, tpar, fault)) return;
        tc_fence_after();
        const uint32_t at = tmem + buf * kAccAt + kSums * half + (uint32_t(32 * (warp & 3)) << 16);
#pragma unroll
        for (int c = 0; c < kSums; c += kRound) {
          float v[kRound];
#pragma unroll
          for (int j = 0; j < kRound; j += 32) tmem_ld32(at + c + j, v + j);
          tmem_ld_wait();
          if (c + kRound >= kSums) {  // the accumulator is free as soon as the last round has it
            tc_fence_before();
            __syncwarp();
            if (lane == 0) arrive_in_cluster(tempty + 8 * buf);
          }
#pragma unroll
          for (int j = 0; j < kRound; ++j) acc[c + j] = fmaf(v[j], f, acc[c + j]);
        }
        buf ^= 1;
        tpar ^= buf == 0;
      }
      __syncwarp();
      if (lane == 0) mbar_arrive(sm.bar(kPbSEmpty + slot));
      if (++slot == kPairSlots) {
        slot = 0;
        spar ^= 1;
      }
    }
    const int cols = min(kSums, p.n - n0), rows = min(32, t.cols - row0);
    if (rows > 0 && cols > 0) {
      const size_t at = size_t(t.row0 + row0) * p.out_row_stride + n0;
      uint8_t* stage = sm.ptr + kOutAt + kOutWarp * warp;
      if (p.out_type == QSFM_BF16)
        store_rows(static_cast<__nv_bfloat16*>(p.out) + at, p.out_row_stride, acc, rows, cols, aligned, stage);
      else if (p.out_type == QSFM_F16)
        store_rows(static_cast<__half*>(p.out) + at, p.out_row_stride, acc, rows, cols, aligned, stage);
      else
        store_rows(static_cast<float*>(p.out) + at, p.out_row_stride, acc, rows, cols, aligned, stage);
    }
  }
}

__global__ void __cluster_dims__(2) __launch_bounds__(kPairThreads, 1)
    pair_kernel(const qsfm_matmul_params p, const PairShape s, int* fault, const __grid_constant__ CUtensorMap amap,
                const __grid_constant__ CUtensorMap wmap) {
  extern __shared__ uint8_t pair_smem[];
  const uint32_t raw = smem_u32(pair_smem);
  MmSmem sm;
  sm.base = (raw + 1023u) & ~1023u;
  sm.ptr = pair_smem + (sm.base - raw);
  sm.bars = kBarAt;
  const int tid = threadIdx.x, warp = tid >> 5;
  const uint32_t rank = cluster_rank();
  int* prefix = reinterpret_cast<int*>(sm.ptr + kPrefixAt);
  if (tid == 0) {
    for (int i = 0; i < kPairStages; ++i) {
      mbar_init(sm.bar(kPbFull + i), 1);
      mbar_init(sm.bar(kPbEmpty + i), 1);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(sm.bar(kPbTFull + i), 1);
      mbar_init(sm.bar(kPbTEmpty + i), 2 * kAddWarps);
    }
    mbar_init(sm.bar(kPbDrain), 1);
    mbar_init(sm.bar(kPbDrain + 1), 1);
    for (int i = 0; i < kPairSlots; ++i) {
      mbar_init(sm.bar(kPbSFull + i), 32);
      mbar_init(sm.bar(kPbSEmpty + i), kAddWarps);
    }
    *sm.abort_flag() = 0;
    fence_mbar_init();
  }
  if (warp == kAddWarps + 1) {  // of both CTAs
    asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_u32(sm.tmem_slot())),
                 "r"(kPairTmem)
                 : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;" ::: "memory");
  }
  grid_dependency_wait();
  grid_launch_dependents();
  if (warp == 0) count_tiles(p, kPairRows, s.col_tiles, prefix, fault);
  tc_fence_before();
  __syncthreads();
  cluster_sync();  // barriers and tensor memory of both CTAs are there
  tc_fence_after();
  const uint32_t tmem = *sm.tmem_slot();
  PairWalk walk;
  walk.prefix = prefix;
  walk.g = 0;
  walk.at = int(blockIdx.x >> 1);
  walk.step = int(gridDim.x >> 1);
  walk.total = prefix[p.groups];
  if (warp < kAddWarps) {
    mm_more_registers<kAddRegs>();
    pair_sum(p, s, sm, walk, rank, tmem, fault);
  } else {
    mm_fewer_registers<kOtherRegs>();
    if (warp == kAddWarps) {
      pair_load(p, s, sm, walk, rank, &amap, &wmap, fault);
    } else if (warp == kAddWarps + 3) {
      pair_scales(p, s, sm, walk, rank, fault);
    } else if (rank == 0) {
      const int odd = warp - kAddWarps - 1;
      pair_issue(p, s, sm, walk, uint32_t(odd), tmem, fault);
      // every MMA issued has completed before tensor memory is freed
      pair_commit(sm.bar(kPbDrain + odd));
      volatile int never = 0;
      if (!mbar_wait_poll(smem_u32(sm.bar(kPbDrain + odd)), 0, &never, kMmTimeoutNs)) atomicOr(fault, QSFM_FAULT_TIMEOUT);
    }
  }
  // after an abort copies may still be on their way into this CTA's shared memory:
  // a millisecond is far more than they take
  __syncwarp();
  if (warp == kAddWarps && *sm.abort_flag())
    for (int i = 0; i < 1000; ++i) __nanosleep(1000);
  __syncwarp();
  tc_fence_before();
  __syncthreads();
  cluster_sync();  // no arrival for the other CTA is on its way, its accumulators are read
  if (warp == kAddWarps + 1) {
    tc_fence_after();
    asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(kPairTmem) : "memory");
  }
}

}  // namespace

cudaError_t launch_matmul_pair(const qsfm_matmul_params& p, int sms, int* fault, cudaStream_t stream) {
  // with fewer registers than the split counts on, the adding warps would wait forever
  static std::atomic<bool> enough{false};
  cudaError_t e;
  if (!enough.load(std::memory_order_relaxed)) {
    cudaFuncAttributes attr;
    if ((e = cudaFuncGetAttributes(&attr, pair_kernel)) != cudaSuccess) return e;
    if (attr.numRegs < kLaunchRegs) return cudaErrorInvalidConfiguration;
    enough.store(true, std::memory_order_relaxed);
  }
  if ((e = cudaFuncSetAttribute(pair_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, int(kPairSmem))) != cudaSuccess)
    return e;
  PairShape s;
  s.kb = (p.k + kMmK - 1) / kMmK;
  s.col_blocks = (p.n + 127) / 128;
  s.col_tiles = (p.n + kPairCols - 1) / kPairCols;
  CUtensorMap amap, wmap;
  if ((e = make_map(p.a, p.k, p.rows, 1, p.a_row_stride, 0, 128, false, &amap)) != cudaSuccess) return e;
  if ((e = make_map(p.w, p.k, p.n, p.groups, p.w_row_stride, p.w_group_stride, kPairCols / 2, true, &wmap)) != cudaSuccess) return e;
  // at most this many tiles: every group but one may add a tile that is not full
  const long long most = ((long long)p.rows / kPairRows + (p.groups < p.rows ? p.groups : p.rows)) * s.col_tiles;
  const int pairs = int(most < sms / 2 ? most : sms / 2);
  return launch_after_predecessor(pair_kernel, dim3(2 * pairs), dim3(kPairThreads), kPairSmem, stream, p, s, fault, amap,
                                  wmap);
}

}  // namespace qsfm
