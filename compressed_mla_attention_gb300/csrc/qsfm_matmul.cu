// Products of e4m3 rows with e4m3 matrices, one fp32 scale per 128 elements of a row
// and per 128 x 128 elements of a matrix, one matrix per group of rows (sm_103a).
//
//   out[m][j] = sum_b a_scale[m][b] w_scale[g][j / 128][b] sum_{k in b} a[m][k] w[g][j][k]
//
// The scales differ from block to block of K, so a block's products (tcgen05.mma
// kind::f8f6f4, fp32 accumulators in tensor memory) are read out, multiplied by their
// two scales and added to sums in registers. This file's kernel is that of few rows (of a
// group, on average; qsfm_matmul_pair.cu has the other). The matrix is the MMA's M side
// (128 of its rows, one scale), the rows of a are its N side (kCols of them at most):
// single tokens waste none of the matrix's stream, and the N of an instruction is what
// the tile has. Tensor-memory lanes are the tile's matrix rows, a thread's sums those of
// one matrix row with rows of a.
//
// Roles: a warp that loads (TMA, 128-byte swizzle), one that issues MMAs, one that
// copies the scales of the tile's rows (cp.async), 4 or 8 that add up and store. A CTA
// walks tiles in turn; the rows of a group fastest, then the matrix's. Where the tiles
// leave SMs without work, a tile's blocks of K are split over a cluster, whose CTAs
// exchange their sums through distributed shared memory.
#include <atomic>

#include "qsfm_matmul_common.cuh"
#ifndef MM_PAIR
#define MM_PAIR (rows > 128)
#endif

namespace qsfm {
namespace {

constexpr int kMmRows = 128;        // matrix rows of a tile
constexpr int kMmScaleSlots = 8;
constexpr int kMmMaxStages = 12;

template <int kCols>
struct MmConfig {
  static constexpr int kLogCols = kCols == 16 ? 4 : kCols == 32 ? 5 : kCols == 64 ? 6 : kCols == 128 ? 7 : 8;
  static constexpr int kEpiWarps = kCols >= 64 ? 8 : 4;
  static constexpr int kWarpCols = kCols >= 64 ? kCols / 2 : kCols;  // columns of an adding warp
  static constexpr int kThreads = 32 * (kEpiWarps + 4);
  // 128 sums a thread and 64 products on their way: registers that the other warps give
  static constexpr bool kShareRegs = kCols == 256;
  static constexpr int kAddRegs = 216, kOtherRegs = 72, kLaunchRegs = 168;
  static_assert(256 * kAddRegs + 128 * kOtherRegs <= 384 * kLaunchRegs, "registers");
  static constexpr int kBoxRows = kCols < 32 ? kCols : 32;  // rows of a per copy
  static constexpr uint32_t kStage = kMmRows * kMmK + kCols * kMmK;
  static constexpr uint32_t kScaleSlot = kCols * 4;
  // after the stages: scale slots, group prefix, barriers
  static constexpr uint32_t kTail = kMmScaleSlots * kScaleSlot + (kMmMaxGroups + 4) * 4 + 512;
  static constexpr int kFit = int((kMmSmemMax - 1024 - kTail) / kStage);
  static constexpr int kStages = kFit < kMmMaxStages ? kFit : kMmMaxStages;
  static constexpr uint32_t kScaleAt = kStages * kStage;
  static constexpr uint32_t kPrefixAt = kScaleAt + kMmScaleSlots * kScaleSlot;
  static constexpr uint32_t kBarAt = (kPrefixAt + (kMmMaxGroups + 4) * 4 + 7) & ~7u;
  static constexpr uint32_t kSmem = kBarAt + 512 + 1024;
  static constexpr uint32_t kTmemCols = 2 * kCols < 32 ? 32 : 2 * kCols;
  static_assert(kSmem <= kMmSmemMax && kCols * kMmRows * 4 <= kScaleAt, "shared memory");
};

// barriers
constexpr int kMbFull = 0, kMbEmpty = kMmMaxStages, kMbSFull = 2 * kMmMaxStages, kMbSEmpty = kMbSFull + kMmScaleSlots,
              kMbTFull = kMbSEmpty + kMmScaleSlots, kMbTEmpty = kMbTFull + 2, kMbDrain = kMbTEmpty + 2,
              kMbCount = kMbDrain + 1;
static_assert(kMbCount * 8 + 8 <= 512, "barriers");

struct MmShape {
  int kb;         // blocks of K
  int col_tiles;  // tiles of the matrix's rows
  int split;      // log2 of the CTAs of a cluster, which share a tile's blocks of K
};

__device__ __forceinline__ void st_cluster(uint32_t addr, float v) {
  asm volatile("st.shared::cluster.f32 [%0], %1;" ::"r"(addr), "f"(v) : "memory");
}

// The CTA's walk over the tiles: prefix[g] tiles lie before group g's.
template <int kCols>
struct MmWalk {
  const int* prefix;
  int g, at, step, total;
  __device__ __forceinline__ bool next(const qsfm_matmul_params& p, const MmShape& s, MmTile& t) {
    if (at >= total) return false;
    while (at >= prefix[g + 1]) ++g;
    int lo, hi;
    bool bad;
    group_rows(p, g, lo, hi, bad);
    const int local = at - prefix[g], row_tiles = (hi - lo + kCols - 1) / kCols;
    const int n = local / row_tiles, m = local - n * row_tiles;
    t.g = g;
    t.n0 = n * kMmRows;
    t.row0 = lo + m * kCols;
    t.cols = min(kCols, hi - t.row0);
    at += step;
    return true;
  }
};

// ------------------------------------------------------------- loads
template <int kCols>
__device__ void mm_load(const qsfm_matmul_params& p, const MmShape& s, const MmSmem& sm, MmWalk<kCols> walk, int b0,
                        int b1, const CUtensorMap* amap, const CUtensorMap* wmap, int* fault) {
  using C = MmConfig<kCols>;
  if ((threadIdx.x & 31) != 0) return;
  uint32_t st = 0, par = 1;
  MmTile t;
  while (walk.next(p, s, t)) {
    const int boxes = (t.cols + C::kBoxRows - 1) / C::kBoxRows;
    const uint32_t bytes = uint32_t(kMmRows + boxes * C::kBoxRows) * kMmK;
    for (int b = b0; b < b1; ++b) {
      if (!mm_wait(sm, kMbEmpty + st, par, fault)) return;
      const uint32_t at = sm.base + st * C::kStage;
      mbar_arrive_expect_tx(sm.bar(kMbFull + st), bytes);
      mm_load_3d(at, wmap, b * kMmK, t.n0, t.g, sm.bar(kMbFull + st));
      for (int i = 0; i < boxes; ++i)
        tma_load_2d(at + kMmRows * kMmK + i * C::kBoxRows * kMmK, amap, b * kMmK, t.row0 + i * C::kBoxRows,
                    sm.bar(kMbFull + st));
      if (++st == C::kStages) {
        st = 0;
        par ^= 1;
      }
    }
  }
}

// ------------------------------------------------------------- MMA issue
template <int kCols>
__device__ void mm_issue(const qsfm_matmul_params& p, const MmShape& s, const MmSmem& sm, MmWalk<kCols> walk, int b0,
                         int b1, uint32_t tmem, int* fault) {
  using C = MmConfig<kCols>;
  uint32_t st = 0, par = 0, buf = 0, tpar = 1;
  MmTile t;
  while (walk.next(p, s, t)) {
    // formats 0 (e4m3) for both operands, as in the bf16 descriptor's f16 form
    const uint32_t idesc = make_idesc_bf16(kMmRows, (t.cols + 15) & ~15, 0, 0, true);
    for (int b = b0; b < b1; ++b) {
      if (!mm_warp_wait(sm, kMbTEmpty + buf, tpar, fault)) return;
      if (!mm_warp_wait(sm, kMbFull + st, par, fault)) return;
      tc_fence_after();
      const uint32_t w = mm_desc(sm.base + st * C::kStage), a = w + ((kMmRows * kMmK) >> 4);
      const uint32_t d = tmem + buf * kCols;
      mma_e4m3<0>(d, w, a, idesc, 0);
      mma_e4m3<2>(d, w, a, idesc, 1);
      mma_e4m3<4>(d, w, a, idesc, 1);
      mma_e4m3<6>(d, w, a, idesc, 1);
      mm_commit(sm.bar(kMbEmpty + st));
      mm_commit(sm.bar(kMbTFull + buf));
      if (++st == C::kStages) {
        st = 0;
        par ^= 1;
      }
      buf ^= 1;
      tpar ^= buf == 0;
    }
  }
}

// ------------------------------------------------------------- scales
template <int kCols>
__device__ void mm_scales(const qsfm_matmul_params& p, const MmShape& s, const MmSmem& sm, MmWalk<kCols> walk, int b0,
                          int b1, int* fault) {
  using C = MmConfig<kCols>;
  const int lane = threadIdx.x & 31;
  uint32_t slot = 0, par = 1;
  MmTile t;
  while (walk.next(p, s, t)) {
    for (int b = b0; b < b1; ++b) {
      if (!mm_warp_wait(sm, kMbSEmpty + slot, par, fault)) return;
      const uint32_t at = sm.base + C::kScaleAt + slot * C::kScaleSlot;
#pragma unroll
      for (int c = lane; c < kCols; c += 32) {
        const bool in = c < t.cols;
        cp_async4(at + 4 * c, p.a_scale + size_t(t.row0 + (in ? c : 0)) * p.a_scale_row_stride +
                                  size_t(b) * p.a_scale_col_stride, in ? 4 : 0);
      }
      cp_async_arrive(sm.bar(kMbSFull + slot));
      if (++slot == kMmScaleSlots) {
        slot = 0;
        par ^= 1;
      }
    }
  }
  asm volatile("cp.async.wait_all;" ::: "memory");
}

// ------------------------------------------------------------- sums and output
// Adds up the blocks b0 .. b1 - 1 of a tile in registers; false after a timeout. A round
// takes up to 64 columns out of tensor memory at once (a load and its wait take 200 cycles
// and more, whatever its size).
template <int kCols>
__device__ __forceinline__ bool mm_add(const qsfm_matmul_params& p, const MmShape& s, const MmSmem& sm, const MmTile& t,
                                       int b0, int b1, uint32_t tmem, uint32_t& buf, uint32_t& tpar, uint32_t& slot,
                                       uint32_t& spar, float (&acc)[MmConfig<kCols>::kWarpCols], int* fault) {
  using C = MmConfig<kCols>;
  constexpr int kN = C::kWarpCols, kRound = kN < 64 ? kN : 64, kPart = kN < 32 ? kN : 32;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int quarter = warp & 3, c0 = (warp >> 2) * kN;
#pragma unroll
  for (int i = 0; i < kN; ++i) acc[i] = 0.f;
  const int live = t.cols - c0;  // columns of this warp
  const float* wsp = p.w_scale + (size_t(t.g) * s.col_tiles + t.n0 / kMmRows) * s.kb;
  // two blocks ahead, into the register that the block of the same parity is done with
  // (a copy from register to register would wait for the load)
  float wsr[2] = {b0 < b1 ? __ldg(wsp + b0) : 0.f, b0 + 1 < b1 ? __ldg(wsp + b0 + 1) : 0.f};
  for (int bb = b0; bb < b1; bb += 2) {
#pragma unroll
   for (int par2 = 0; par2 < 2; ++par2) {
    const int b = bb + par2;
    if (b >= b1) break;
    const float ws = wsr[par2];
    if (b + 2 < b1) wsr[par2] = __ldg(wsp + b + 2);
    if (!mm_warp_wait(sm, kMbSFull + slot, spar, fault)) return false;
    if (!mm_warp_wait(sm, kMbTFull + buf, tpar, fault)) return false;
    tc_fence_after();
    const float4* sc = reinterpret_cast<const float4*>(sm.ptr + C::kScaleAt + slot * C::kScaleSlot) + c0 / 4;
    const uint32_t at = tmem + buf * kCols + c0 + (uint32_t(32 * quarter) << 16);
#pragma unroll
    for (int c = 0; c < kN; c += kRound) {
      float v[kRound];
#pragma unroll
      for (int h = 0; h < kRound; h += kPart)
        if (c + h < live) {
          if constexpr (kPart == 32) tmem_ld32(at + c + h, v + h);
          else tmem_ld16(at + c + h, v + h);
        }
      tmem_ld_wait();
      if (c + kRound >= kN) {  // the accumulator is free as soon as the last round has it
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(sm.bar(kMbTEmpty + buf));
      }
#pragma unroll
      for (int h = 0; h < kRound; h += kPart)
        if (c + h < live) {
#pragma unroll
          for (int i = h; i < h + kPart; i += 4) {
            const float4 f = sc[(c + i) / 4];
            mm_fma2(acc[c + i], acc[c + i + 1], v[i], v[i + 1], f.x * ws, f.y * ws);
            mm_fma2(acc[c + i + 2], acc[c + i + 3], v[i + 2], v[i + 3], f.z * ws, f.w * ws);
          }
        }
    }
    __syncwarp();
    if (lane == 0) mbar_arrive(sm.bar(kMbSEmpty + slot));
    buf ^= 1;
    tpar ^= buf == 0;
    if (++slot == kMmScaleSlots) {
      slot = 0;
      spar ^= 1;
    }
   }
  }
  return true;
}

template <int kCols>
__device__ void mm_sum(const qsfm_matmul_params& p, const MmShape& s, const MmSmem& sm, MmWalk<kCols> walk, int b0,
                       int b1, uint32_t tmem, int* fault) {
  using C = MmConfig<kCols>;
  constexpr int kN = C::kWarpCols;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int row = 32 * (warp & 3) + lane, c0 = (warp >> 2) * kN;
  uint32_t buf = 0, tpar = 0, slot = 0, spar = 0;
  MmTile t;
  float acc[kN];
  if (s.split == 0) {
    while (walk.next(p, s, t)) {
      if (!mm_add<kCols>(p, s, sm, t, b0, b1, tmem, buf, tpar, slot, spar, acc, fault)) return;
      if (t.n0 + row < p.n) {
#pragma unroll
        for (int c = 0; c < kN; ++c)
          if (c0 + c < t.cols) mm_store(p, size_t(t.row0 + c0 + c) * p.out_row_stride + t.n0 + row, acc[c]);
      }
    }
    return;
  }
  // The cluster's one tile: CTA r adds up the columns r w .. r w + w - 1 of all, w = kCols /
  // CTAs, in the order of the CTAs. Their sums take the place of the operands, which every
  // CTA of the cluster is through with at the first barrier.
  bool ok = walk.next(p, s, t);
  if (ok) ok = mm_add<kCols>(p, s, sm, t, b0, b1, tmem, buf, tpar, slot, spar, acc, fault);
  const uint32_t rank = cluster_rank();
  const int shift = C::kLogCols - s.split, w = 1 << shift;
  cluster_sync();
  if (ok) {
#pragma unroll
    for (int c = 0; c < kN; ++c) {
      const int col = c0 + c;
      if (col < t.cols)
        st_cluster(in_cta(sm.base + 4 * (((rank << shift) + (col & (w - 1))) * kMmRows + row), uint32_t(col >> shift)), acc[c]);
    }
  }
  cluster_sync();
  if (!ok || t.n0 + row >= p.n) return;
  const float* sums = reinterpret_cast<const float*>(sm.ptr) + row;
  for (int c = warp >> 2; c < w; c += C::kEpiWarps / 4) {
    const int col = int(rank << shift) + c;
    if (col >= t.cols) break;
    float v = sums[c * kMmRows];
    for (int r = 1; r < 1 << s.split; ++r) v += sums[((r << shift) + c) * kMmRows];
    mm_store(p, size_t(t.row0 + col) * p.out_row_stride + t.n0 + row, v);
  }
}

template <int kCols>
__global__ void __launch_bounds__(MmConfig<kCols>::kThreads, 1)
    matmul_kernel(const qsfm_matmul_params p, const MmShape s, int* fault, const __grid_constant__ CUtensorMap amap,
                  const __grid_constant__ CUtensorMap wmap) {
  using C = MmConfig<kCols>;
  extern __shared__ uint8_t mm_smem[];
  const uint32_t raw = smem_u32(mm_smem);
  MmSmem sm;
  sm.base = (raw + 1023u) & ~1023u;
  sm.ptr = mm_smem + (sm.base - raw);
  sm.bars = C::kBarAt;
  const int tid = threadIdx.x, warp = tid >> 5;
  int* prefix = reinterpret_cast<int*>(sm.ptr + C::kPrefixAt);
  if (tid == 0) {
    for (int i = 0; i < C::kStages; ++i) {
      mbar_init(sm.bar(kMbFull + i), 1);
      mbar_init(sm.bar(kMbEmpty + i), 1);
    }
    for (int i = 0; i < kMmScaleSlots; ++i) {
      mbar_init(sm.bar(kMbSFull + i), 32);
      mbar_init(sm.bar(kMbSEmpty + i), C::kEpiWarps);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(sm.bar(kMbTFull + i), 1);
      mbar_init(sm.bar(kMbTEmpty + i), C::kEpiWarps);
    }
    mbar_init(sm.bar(kMbDrain), 1);
    *sm.abort_flag() = 0;
    fence_mbar_init();
  }
  if (warp == C::kEpiWarps + 1) tmem_alloc(sm.tmem_slot(), C::kTmemCols);
  grid_dependency_wait();
  grid_launch_dependents();
  if (warp == 0) count_tiles(p, kCols, s.col_tiles, prefix, fault);
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *sm.tmem_slot();
  MmWalk<kCols> walk;
  walk.prefix = prefix;
  walk.g = 0;
  walk.at = int(blockIdx.x >> s.split);
  walk.step = int(gridDim.x >> s.split);
  walk.total = prefix[p.groups];
  const int part = int(blockIdx.x) & ((1 << s.split) - 1);
  const int b0 = int(int64_t(s.kb) * part >> s.split), b1 = int(int64_t(s.kb) * (part + 1) >> s.split);
  if constexpr (C::kShareRegs) {
    if (warp < C::kEpiWarps) mm_more_registers<C::kAddRegs>();
    else mm_fewer_registers<C::kOtherRegs>();
  }
  if (warp < C::kEpiWarps) {
    mm_sum<kCols>(p, s, sm, walk, b0, b1, tmem, fault);
  } else if (warp == C::kEpiWarps) {
    mm_load<kCols>(p, s, sm, walk, b0, b1, &amap, &wmap, fault);
  } else if (warp == C::kEpiWarps + 1) {
    mm_issue<kCols>(p, s, sm, walk, b0, b1, tmem, fault);
    // every MMA issued has completed before tensor memory is freed
    mm_commit(sm.bar(kMbDrain));
    volatile int never = 0;
    if (!mbar_wait_poll(smem_u32(sm.bar(kMbDrain)), 0, &never, kMmTimeoutNs)) atomicOr(fault, QSFM_FAULT_TIMEOUT);
  } else if (warp == C::kEpiWarps + 2) {
    mm_scales<kCols>(p, s, sm, walk, b0, b1, fault);
  }
  __syncwarp();
  if (s.split > 0 && warp >= C::kEpiWarps) {  // (the adding warps' are in mm_sum)
    cluster_sync();
    cluster_sync();
  }
  // after an abort copies may still be on their way into this CTA's shared memory:
  // a millisecond is far more than they take
  if (warp == C::kEpiWarps && *sm.abort_flag())
    for (int i = 0; i < 1000; ++i) __nanosleep(1000);
  __syncwarp();
  tc_fence_before();
  __syncthreads();
  if (warp == C::kEpiWarps + 1) {
    tc_fence_after();
    tmem_dealloc(tmem, C::kTmemCols);
  }
}

// ------------------------------------------------------------- host side
template <int kCols>
cudaError_t launch_cols(const qsfm_matmul_params& p, const MmShape& s, int sms, int* fault, cudaStream_t stream) {
  using C = MmConfig<kCols>;
  cudaError_t e = cudaFuncSetAttribute(matmul_kernel<kCols>, cudaFuncAttributeMaxDynamicSharedMemorySize, int(C::kSmem));
  if (e != cudaSuccess) return e;
  if constexpr (C::kShareRegs) {
    // with fewer registers than the split counts on, the adding warps would wait forever
    static std::atomic<bool> enough{false};
    if (!enough.load(std::memory_order_relaxed)) {
      cudaFuncAttributes attr;
      if ((e = cudaFuncGetAttributes(&attr, matmul_kernel<kCols>)) != cudaSuccess) return e;
      if (attr.numRegs < C::kLaunchRegs) return cudaErrorInvalidConfiguration;
      enough.store(true, std::memory_order_relaxed);
    }
  }
  CUtensorMap amap, wmap;
  if ((e = make_map(p.a, p.k, p.rows, 1, p.a_row_stride, 0, C::kBoxRows, false, &amap)) != cudaSuccess) return e;
  if ((e = make_map(p.w, p.k, p.n, p.groups, p.w_row_stride, p.w_group_stride, kMmRows, true, &wmap)) != cudaSuccess)
    return e;
  // at most this many tiles: every group but one may add a tile that is not full
  const long long most = p.cu_rows == nullptr
                             ? (long long)((p.rows + kCols - 1) / kCols) * s.col_tiles
                             : ((long long)p.rows / kCols + (p.groups < p.rows ? p.groups : p.rows)) * s.col_tiles;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(s.split > 0 ? unsigned(most << s.split) : unsigned(most < sms ? most : sms));
  cfg.blockDim = dim3(C::kThreads);
  cfg.dynamicSmemBytes = C::kSmem;
  cfg.stream = stream;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = 1u << s.split;
  attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = s.split > 0 ? 2 : 1;
  return cudaLaunchKernelEx(&cfg, matmul_kernel<kCols>, p, s, fault, amap, wmap);
}

}  // namespace

cudaError_t launch_matmul(const qsfm_matmul_params& p, int* fault, cudaStream_t stream) {
  int dev = 0, sms = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  if ((e = cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev)) != cudaSuccess) return e;
  MmShape s;
  s.kb = (p.k + kMmK - 1) / kMmK;
  s.col_tiles = (p.n + kMmRows - 1) / kMmRows;
  s.split = 0;
  const int rows = (p.rows + p.groups - 1) / p.groups;  // of a group, on average
  if (MM_PAIR) return launch_matmul_pair(p, sms, fault, stream);
  int cols = rows <= 16 ? 16 : rows <= 32 ? 32 : rows <= 64 ? 64 : rows <= 128 ? 128 : 256;
#ifdef MM_COLS
  cols = MM_COLS;
#endif
  // the tiles of one group are known here: where they leave SMs without work, the
  // blocks of K are split, down to two blocks a CTA
  if (p.cu_rows == nullptr) {
    const long long tiles = (long long)((p.rows + cols - 1) / cols) * s.col_tiles;
    while (s.split < 3 && (tiles << (s.split + 1)) <= sms && s.kb >= 4 << s.split) ++s.split;
#ifdef MM_SPLIT
    s.split = MM_SPLIT;
#endif
  }
  switch (cols) {
    case 16: return launch_cols<16>(p, s, sms, fault, stream);
    case 32: return launch_cols<32>(p, s, sms, fault, stream);
    case 64: return launch_cols<64>(p, s, sms, fault, stream);
    case 128: return launch_cols<128>(p, s, sms, fault, stream);
    default: return launch_cols<256>(p, s, sms, fault, stream);
  }
}

}  // namespace qsfm
