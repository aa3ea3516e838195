// Products of e4m3 rows with e4m3 matrices, one fp32 scale per 128 elements of a row
// and per 128 x 128 elements of a matrix, one matrix per group of rows (sm_103a).
//
//   out[m][j] = sum_b a_scale[m][b] w_scale[g][j / 128][b] sum_{k in b} a[m][k] w[g][j][k]
//
// The scales differ from block to block of K, so a block's products (tcgen05.mma
// kind::f8f6f4, fp32 accumulators in tensor memory) are read out, multiplied by their
// two scales and added to sums in registers. The matrix is the MMA's M side (128 of its
// rows, one scale), the rows of a are its N side (kCols of them at most): single tokens
// waste none of the matrix's stream, and the N of an instruction is what the tile has.
// The tile's matrix rows are tensor-memory lanes, a thread's sums those of one matrix
// row with every row of a.
//
// Roles: a warp that loads (TMA, 128-byte swizzle), one that issues MMAs, one that
// copies the scales of the tile's rows (cp.async), 4 or 8 that add up and store. A
// CTA walks tiles in turn; the rows of a group of rows fastest, then the matrix's.
#include <cuda.h>
#include <cudaTypedefs.h>
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include <mutex>

#include "qsfm_device.cuh"
#include "qsfm_internal.h"

namespace qsfm {
namespace {

constexpr int kMmRows = 128;        // matrix rows of a tile
constexpr int kMmK = 128;           // bytes of K per stage: one block of scales
constexpr int kMmMaxGroups = 1024;
constexpr long long kMmMaxTiles = (1ll << 30) + 1;  // counted at most
constexpr int kMmScaleSlots = 8;
constexpr int kMmMaxStages = 12;
constexpr uint64_t kMmTimeoutNs = 1000000000ull;
constexpr uint32_t kMmSmemMax = 227 * 1024;

template <int kCols>
struct MmConfig {
  static constexpr int kEpiWarps = kCols > 128 ? 8 : 4;
  static constexpr int kWarpCols = kCols > 128 ? kCols / 2 : kCols;  // columns of an adding warp
  static constexpr int kThreads = 32 * (kEpiWarps + 3);
  static constexpr int kBoxRows = kCols < 32 ? kCols : 32;           // rows of a per copy
  static constexpr uint32_t kStage = kMmRows * kMmK + kCols * kMmK;
  static constexpr uint32_t kScaleSlot = kCols * 4;
  // after the stages: scale slots, group prefix, barriers, the rest
  static constexpr uint32_t kTail = kMmScaleSlots * kScaleSlot + (kMmMaxGroups + 4) * 4 + 512;
  static constexpr int kFit = int((kMmSmemMax - 1024 - kTail) / kStage);
  static constexpr int kStages = kFit < kMmMaxStages ? kFit : kMmMaxStages;
  static constexpr uint32_t kScaleAt = kStages * kStage;
  static constexpr uint32_t kPrefixAt = kScaleAt + kMmScaleSlots * kScaleSlot;
  static constexpr uint32_t kBarAt = (kPrefixAt + (kMmMaxGroups + 4) * 4 + 7) & ~7u;
  static constexpr uint32_t kSmem = kBarAt + 512 + 1024;
  static constexpr uint32_t kTmemCols = 2 * kCols < 32 ? 32 : 2 * kCols;
  static_assert(kSmem <= kMmSmemMax, "shared memory");
};

// barriers
constexpr int kMbFull = 0, kMbEmpty = kMmMaxStages, kMbSFull = 2 * kMmMaxStages, kMbSEmpty = kMbSFull + kMmScaleSlots,
              kMbTFull = kMbSEmpty + kMmScaleSlots, kMbTEmpty = kMbTFull + 2, kMbDrain = kMbTEmpty + 2,
              kMbCount = kMbDrain + 1;
static_assert(kMbCount * 8 + 16 <= 512, "barriers");

struct MmShape {
  int kb;        // blocks of K
  int col_tiles; // tiles of the matrix's rows
};

struct MmSmem {
  uint32_t base;
  uint8_t* ptr;
  uint32_t bars;  // offset of the barriers
  __device__ uint64_t* bar(int i) const { return reinterpret_cast<uint64_t*>(ptr + bars) + i; }
  __device__ uint32_t* tmem_slot() const { return reinterpret_cast<uint32_t*>(ptr + bars + kMbCount * 8); }
  __device__ volatile int* abort_flag() const { return reinterpret_cast<volatile int*>(ptr + bars + kMbCount * 8 + 4); }
};

__device__ __forceinline__ bool mm_wait(const MmSmem& sm, int bar, uint32_t parity, int* fault) {
  if (mbar_wait_bounded(sm.bar(bar), parity, sm.abort_flag(), kMmTimeoutNs)) return true;
  if (!*sm.abort_flag()) {
    *sm.abort_flag() = 1;
    atomicOr(fault, QSFM_FAULT_TIMEOUT);
  }
  return false;
}

// Every lane waits (on an open barrier one test), the warp goes on together.
__device__ __forceinline__ bool mm_warp_wait(const MmSmem& sm, int bar, uint32_t parity, int* fault) {
  const bool ok = mm_wait(sm, bar, parity, fault);
  return __all_sync(0xffffffffu, ok) != 0;
}

__device__ __forceinline__ void mm_load_3d(uint32_t dst, const void* tmap, int x, int y, int z, uint64_t* bar) {
  asm volatile(
      "cp.async.bulk.tensor.3d.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
      " [%0], [%1, {%2, %3, %4}], [%5];" ::"r"(dst),
      "l"(reinterpret_cast<uint64_t>(tmap)), "r"(x), "r"(y), "r"(z), "r"(smem_u32(bar))
      : "memory");
}

// 4 bytes to shared memory without a register, zeros where `bytes` is 0.
__device__ __forceinline__ void cp_async4(uint32_t dst, const void* src, uint32_t bytes) {
  asm volatile("cp.async.ca.shared.global [%0], [%1], 4, %2;" ::"r"(dst), "l"(src), "r"(bytes) : "memory");
}
// One of the barrier's arrivals, once the thread's copies so far have landed.
__device__ __forceinline__ void cp_async_arrive(uint64_t* bar) {
  asm volatile("cp.async.mbarrier.arrive.noinc.shared::cta.b64 [%0];" ::"r"(smem_u32(bar)) : "memory");
}

// D (+)= A B^T of 32 e4m3 of K, operands K-major with the 128-byte swizzle (8-row groups
// of 1 KB). The whole warp runs the loop around it and one elected lane issues, so the
// descriptors stay in uniform registers.
constexpr uint32_t kMmDescHigh = (1024u >> 4) | (1u << 14) | (2u << 29);  // group stride, version, swizzle
template <uint32_t kOff>
__device__ __forceinline__ void mma_e4m3(uint32_t d, uint32_t a, uint32_t b, uint32_t idesc, uint32_t accumulate) {
  asm volatile(
      "{\n .reg .pred p, e;\n .reg .b32 x, y;\n .reg .b64 a, b;\n add.u32 x, %1, %6;\n add.u32 y, %2, %6;\n"
      " mov.b64 a, {x, %5};\n mov.b64 b, {y, %5};\n"
      " setp.ne.b32 p, %4, 0;\n elect.sync _|e, 0xffffffff;\n"
      " @e tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], a, b, %3, p;\n}" ::"r"(d),
      "r"(a), "r"(b), "r"(idesc), "r"(accumulate), "n"(kMmDescHigh), "n"(kOff)
      : "memory");
}
__device__ __forceinline__ void mm_commit(uint64_t* bar) {
  asm volatile(
      "{\n .reg .pred e;\n elect.sync _|e, 0xffffffff;\n"
      " @e tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];\n}" ::"r"(smem_u32(bar))
      : "memory");
}
__device__ __forceinline__ uint32_t mm_desc(uint32_t saddr) { return ((saddr >> 4) & 0x3FFFu) | ((16u >> 4) << 16); }

// (s0, s1) += (c0, c1) * (f0, f1), each as fmaf rounds.
__device__ __forceinline__ void mm_fma2(float& s0, float& s1, float c0, float c1, float f0, float f1) {
  asm("{\n .reg .b64 a, b, d;\n mov.b64 a, {%2, %3};\n mov.b64 b, {%4, %5};\n mov.b64 d, {%0, %1};\n"
      " fma.rn.f32x2 d, a, b, d;\n mov.b64 {%0, %1}, d;\n}"
      : "+f"(s0), "+f"(s1)
      : "f"(c0), "f"(c1), "f"(f0), "f"(f1));
}

// One tile: rows row0 .. row0 + cols - 1 of a, matrix rows n0 .. of group g.
struct MmTile {
  int g, n0, row0, cols;
};

// Rows of group g, cut to what there is.
__device__ __forceinline__ void group_rows(const qsfm_matmul_params& p, int g, int& lo, int& hi, bool& bad) {
  if (p.cu_rows == nullptr) {
    lo = 0;
    hi = p.rows;
    bad = false;
    return;
  }
  const int a = __ldg(p.cu_rows + g), b = __ldg(p.cu_rows + g + 1);
  bad = a < 0 || b < a || b > p.rows;
  lo = min(max(a, 0), p.rows);
  hi = max(lo, min(b, p.rows));
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
__device__ __forceinline__ void mm_store(const qsfm_matmul_params& p, size_t at, float v) {
  if (p.out_type == QSFM_BF16) static_cast<__nv_bfloat16*>(p.out)[at] = __float2bfloat16(v);
  else if (p.out_type == QSFM_F16) static_cast<__half*>(p.out)[at] = __float2half(v);
  else static_cast<float*>(p.out)[at] = v;
}

template <int kCols>
__device__ void mm_sum(const qsfm_matmul_params& p, const MmShape& s, const MmSmem& sm, MmWalk<kCols> walk, int b0,
                       int b1, uint32_t tmem, int* fault) {
  using C = MmConfig<kCols>;
  constexpr int kN = C::kWarpCols;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int quarter = warp & 3, c0 = (warp >> 2) * kN;
  uint32_t buf = 0, tpar = 0, slot = 0, spar = 0;
  MmTile t;
  while (walk.next(p, s, t)) {
    float acc[kN];
#pragma unroll
    for (int i = 0; i < kN; ++i) acc[i] = 0.f;
    const int live = t.cols - c0;  // columns of this warp
    const float* wsp = p.w_scale + (size_t(t.g) * s.col_tiles + t.n0 / kMmRows) * s.kb;
    float ws = b0 < b1 ? __ldg(wsp + b0) : 0.f;
    for (int b = b0; b < b1; ++b) {
      const float wnext = b + 1 < b1 ? __ldg(wsp + b + 1) : 0.f;
      if (!mm_warp_wait(sm, kMbSFull + slot, spar, fault)) return;
      if (!mm_warp_wait(sm, kMbTFull + buf, tpar, fault)) return;
      tc_fence_after();
      const float4* sc = reinterpret_cast<const float4*>(sm.ptr + C::kScaleAt + slot * C::kScaleSlot) + c0 / 4;
      const uint32_t at = tmem + buf * kCols + c0 + (uint32_t(32 * quarter) << 16);
#pragma unroll
      for (int c = 0; c < kN; c += 16) {
        if (c < live) {
          float v[16];
          tmem_ld16(at + c, v);
          tmem_ld_wait();
#pragma unroll
          for (int i = 0; i < 16; i += 4) {
            const float4 f = sc[(c + i) / 4];
            mm_fma2(acc[c + i], acc[c + i + 1], v[i], v[i + 1], f.x * ws, f.y * ws);
            mm_fma2(acc[c + i + 2], acc[c + i + 3], v[i + 2], v[i + 3], f.z * ws, f.w * ws);
          }
        }
      }
      tc_fence_before();
      __syncwarp();
      if (lane == 0) {
        mbar_arrive(sm.bar(kMbTEmpty + buf));
        mbar_arrive(sm.bar(kMbSEmpty + slot));
      }
      ws = wnext;
      buf ^= 1;
      tpar ^= buf == 0;
      if (++slot == kMmScaleSlots) {
        slot = 0;
        spar ^= 1;
      }
    }
    const int n = t.n0 + 32 * quarter + lane;
    if (n < p.n) {
#pragma unroll
      for (int c = 0; c < kN; ++c)
        if (c < live) mm_store(p, size_t(t.row0 + c0 + c) * p.out_row_stride + n, acc[c]);
    }
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
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
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
  if (warp == 0) {  // tiles before each group
    long long run = 0;  // overlapping groups of a bad cu_rows may count more than there can be
    const auto cut = [](long long v) { return int(v < kMmMaxTiles ? v : kMmMaxTiles); };
    for (int g0 = 0; g0 < p.groups; g0 += 32) {
      long long n = 0;
      if (g0 + lane < p.groups) {
        int lo, hi;
        bool bad;
        group_rows(p, g0 + lane, lo, hi, bad);
        if (bad && blockIdx.x == 0) atomicOr(fault, QSFM_FAULT_GROUP_ROWS);
        n = (long long)((hi - lo + kCols - 1) / kCols) * s.col_tiles;
      }
      long long sum = n;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const long long up = __shfl_up_sync(0xffffffffu, sum, o);
        if (lane >= o) sum += up;
      }
      if (g0 + lane < p.groups) prefix[g0 + lane] = cut(run + sum - n);
      run += __shfl_sync(0xffffffffu, sum, 31);
    }
    if (lane == 0) prefix[p.groups] = cut(run);
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *sm.tmem_slot();
  MmWalk<kCols> walk;
  walk.prefix = prefix;
  walk.g = 0;
  walk.at = int(blockIdx.x);
  walk.step = int(gridDim.x);
  walk.total = prefix[p.groups];
  const int b0 = 0, b1 = s.kb;
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
  } else {
    mm_scales<kCols>(p, s, sm, walk, b0, b1, fault);
  }
  // after an abort copies may still be on their way into this CTA's shared memory:
  // a millisecond is far more than they take
  __syncwarp();
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
PFN_cuTensorMapEncodeTiled_v12000 tensor_map_encoder() {
  static PFN_cuTensorMapEncodeTiled_v12000 encode = nullptr;
  static std::once_flag once;
  std::call_once(once, [] {
    cudaDriverEntryPointQueryResult qres;
    void* fn = nullptr;
    if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &fn, 12000, cudaEnableDefault, &qres) ==
            cudaSuccess &&
        qres == cudaDriverEntryPointSuccess)
      encode = reinterpret_cast<PFN_cuTensorMapEncodeTiled_v12000>(fn);
  });
  return encode;
}

// Bytes [planes, rows, k] in boxes of box_rows x 128, what lies outside read as zero.
// (A stride of a dimension of length 1 is not used: the encoder still wants it to be a
// multiple of 16 that is not below the extent within.)
cudaError_t make_map(const void* base, int k, int rows, int planes, long long row_stride, long long plane_stride,
                     int box_rows, bool is3d, CUtensorMap* map) {
  const auto encode = tensor_map_encoder();
  if (encode == nullptr) return cudaErrorNotSupported;
  if (rows <= 1) row_stride = (k + 15) & ~15;
  if (planes <= 1) plane_stride = row_stride * rows;
  const cuuint64_t dims[3] = {cuuint64_t(k), cuuint64_t(rows), cuuint64_t(planes)};
  const cuuint64_t strides[2] = {cuuint64_t(row_stride), cuuint64_t(plane_stride)};
  const cuuint32_t box[3] = {kMmK, cuuint32_t(box_rows), 1};
  const cuuint32_t estr[3] = {1, 1, 1};
  const CUresult r = encode(map, CU_TENSOR_MAP_DATA_TYPE_UINT8, is3d ? 3 : 2, const_cast<void*>(base), dims, strides,
                            box, estr, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
                            CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
  return r == CUDA_SUCCESS ? cudaSuccess : cudaErrorInvalidValue;
}

template <int kCols>
cudaError_t launch_cols(const qsfm_matmul_params& p, const MmShape& s, int sms, int* fault, cudaStream_t stream) {
  using C = MmConfig<kCols>;
  cudaError_t e = cudaFuncSetAttribute(matmul_kernel<kCols>, cudaFuncAttributeMaxDynamicSharedMemorySize, int(C::kSmem));
  if (e != cudaSuccess) return e;
  CUtensorMap amap, wmap;
  if ((e = make_map(p.a, p.k, p.rows, 1, p.a_row_stride, 0, C::kBoxRows, false, &amap)) != cudaSuccess) return e;
  if ((e = make_map(p.w, p.k, p.n, p.groups, p.w_row_stride, p.w_group_stride, kMmRows, true, &wmap)) != cudaSuccess)
    return e;
  // at most this many tiles: every group but one may add a tile that is not full
  const long long most = ((long long)p.rows / kCols + (p.groups < p.rows ? p.groups : p.rows)) * s.col_tiles;
  const int grid = int(most < sms ? most : sms);
  return launch_after_predecessor(matmul_kernel<kCols>, dim3(grid), dim3(C::kThreads), C::kSmem, stream, p, s, fault,
                                  amap, wmap);
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
  const int rows = (p.rows + p.groups - 1) / p.groups;  // of a group, on average
  if (rows <= 16) return launch_cols<16>(p, s, sms, fault, stream);
  if (rows <= 32) return launch_cols<32>(p, s, sms, fault, stream);
  if (rows <= 64) return launch_cols<64>(p, s, sms, fault, stream);
  if (rows <= 128) return launch_cols<128>(p, s, sms, fault, stream);
  return launch_cols<256>(p, s, sms, fault, stream);
}

}  // namespace qsfm
