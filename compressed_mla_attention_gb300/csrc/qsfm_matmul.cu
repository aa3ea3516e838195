// Products of e4m3 rows with e4m3 matrices, one fp32 scale per 128 elements of a row
// and per 128 x 128 elements of a matrix, one matrix per group of rows (sm_103a).
//
//   out[m][j] = sum_b a_scale[m][b] w_scale[g][j / 128][b] sum_{k in b} a[m][k] w[g][j][k]
//
// The scales differ from block to block of K, so a block's products (tcgen05.mma
// kind::f8f6f4, fp32 accumulators in tensor memory) are read out, multiplied by their
// two scales and added to sums in registers. Rows of a are the tensor-memory lanes: a
// thread's 128 sums are those of one row with 128 matrix rows, which have one scale, so a
// block's factor is one number a thread, and fp32's product of the two scales: taken one after
// the other where that leaves the normal numbers, they cost 8192 x 4096 x 32768 another 6 to 11%
// (the adding loop has no register left for a second way).
//
// Three kernels, by the estimate of their time at MmTimes: tiles of 256 rows of a by 256
// matrix rows of a pair of CTAs (cta_group::2), each of which loads its own 128 rows of a
// and half of the matrix's, 32 KB a block of K instead of 48; 128 by 256 of a CTA, whose
// clusters take more parts; and 128 by 128, of which there are more and whose sums are
// fewer to join. (2048 x 4096 x 4096: 34.2, 36.0, 51.5 us; 256 x 4096 x 32768 in parts:
// 48.6, 41.7, 54.2; 128 x 4096 x 4096 in parts: 15.1, 13.0, 10.4.) With few rows the
// matrix's bytes are what a product has to read, four stages of 16 or 32 KB a CTA on their
// way; rows of a that are not there are not loaded, and warps without rows do not add.
//
// Per CTA: a warp that loads (TMA, 128-byte swizzle), two that issue MMAs in turn (of a
// pair's first CTA alone), one that copies scales, eight that add up and store. A block's
// MMAs take 512 cycles; meanwhile the eight warps read the previous one's products out of
// tensor memory and add them up. What it took (cycles a block of a pair, K = 8192):
//  * a release of an accumulator at the cluster's scope waits for all the thread's memory
//    operations: 2800 -> 1250 without;
//  * single FMAs instead of pairs (fma.rn.f32x2: 64 a thread took longer than 128): 960;
//  * scales through shared memory, some blocks at a time, instead of 4-byte loads: 770;
//  * a second warp that issues: 715.
// What is left is the way of an accumulator: commit, products read, release, next MMAs,
// some 1300 cycles over the two that tensor memory has room for. 8192 x 8192 x 8192 takes
// 380 us (2.9 PFLOP/s); in a loop the GPU is at its power limit and takes 420, a library's
// product of the same codes without scales 330. Slower or no faster: tiles of 192 matrix
// rows, two MMAs of 128 matrix rows each, 32 products of a thread at a time, six stages,
// a test of the next accumulator ahead of time, waits by one lane of a warp.
//
// A CTA (or pair) walks tiles in turn, eight row tiles of a group before the next of the
// matrix's. Where the tiles of one group leave SMs without work, a tile's blocks of K are
// split over a cluster, whose CTAs exchange their sums through distributed shared memory
// and add them in the order of the CTAs (1 x 4096 x 4096: 8.0 us in four parts, 13.8 in
// one).
#include <cuda.h>
#include <cudaTypedefs.h>
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include <atomic>
#include <climits>
#include <cmath>
#include <mutex>

#include "qsfm_device.cuh"
#include "qsfm_divide.cuh"
#include "qsfm_internal.h"

namespace qsfm {
namespace {

constexpr int kMmK = 128;         // bytes of K per stage: one block of scales
constexpr int kChunk = 16;        // columns that a part of a split tile joins at a time
constexpr int kChunkBytes = kChunk * 128 * 4;
constexpr int kBlockTiles = 8;    // row tiles that are walked before the next of the matrix's
constexpr long long kMaxTiles = kMaxMatmulTiles + 1;  // counted at most
constexpr int kAddWarps = 8;
constexpr int kMmThreads = 32 * (kAddWarps + 4);
constexpr int kAddRegs = 224, kOtherRegs = 56, kLaunchRegs = 168;
static_assert(256 * kAddRegs + 128 * kOtherRegs <= kMmThreads * kLaunchRegs, "registers");
constexpr int kSlots = 4, kSlotBlocks = 4;  // scales of 4 blocks of K at a time
constexpr uint32_t kSlotBlock = 512 + 16;   // 128 rows' scales, one of the matrix's for each half
constexpr uint32_t kOutPart = 2048;         // of an adding warp: 32 rows x 64 bytes on their way out
constexpr uint32_t kOutBox = 4096;          // 32 rows x 128 bytes, a copy's
constexpr uint64_t kMmTimeoutNs = 1000000000ull;

// Tiles of 128 kCtas_ rows of a by kCols_ matrix rows.
template <int kCtas_, int kCols_>
struct Mm {
  static constexpr int kCtas = kCtas_, kCols = kCols_, kRows = 128 * kCtas;
  static constexpr int kSums = kCols / 2;  // of an adding thread
  static constexpr int kRound = 64;        // products of a thread on their way from tensor memory
  static constexpr uint32_t kTmem = 2 * kCols;                             // two accumulators
  static constexpr uint32_t kABytes = 128 * kMmK, kWRows = kCols / kCtas;  // a CTA's
  static constexpr uint32_t kStage = kABytes + kWRows * kMmK;
  static constexpr int kStages = 4;
  // two boxes of output an adding warp, where there is room
  static constexpr bool kBoxes = kStages * kStage + kAddWarps * 2 * kOutBox <= 200 * 1024;
  static constexpr uint32_t kOutWarp = kBoxes ? 2 * kOutBox : kOutPart;
  static_assert(kStages % 2 == 0, "an issuing warp's stages are every other one");
  static constexpr uint32_t kOutAt = kStages * kStage, kScaleAt = kOutAt + kAddWarps * kOutWarp;
  // where a split tile's joined sums are on their way out, behind the parts' sums
  static constexpr uint32_t kJoinedAt = kScaleAt - kAddWarps * kOutPart;
  static constexpr uint32_t kPrefixAt = kScaleAt + kSlots * kSlotBlocks * kSlotBlock;
  static constexpr uint32_t kBarAt = (kPrefixAt + (kMaxMatmulGroups + 4) * 4 + 7) & ~7u;
  static constexpr uint32_t kSmem = kBarAt + 256 + 1024;
  static_assert(kSmem <= 227 * 1024, "shared memory");
};

// barriers; of a pair, those marked * are used in the first CTA alone
constexpr int kMaxStages = 4;
constexpr int kBFull = 0 /* * both CTAs' copies */, kBEmpty = kMaxStages, kBTFull = 2 * kMaxStages,
              kBTEmpty = kBTFull + 2 /* * both CTAs' adding warps */, kBDrain = kBTEmpty + 2 /* * of each issuing warp */,
              kBSFull = kBDrain + 2, kBSEmpty = kBSFull + kSlots, kBCount = kBSEmpty + kSlots;
static_assert(kBCount * 8 + 8 <= 256 && kBCount <= 32, "barriers");

struct MmShape {
  int kb;          // blocks of K
  int col_tiles;   // tiles of the matrix's rows
  int col_blocks;  // scales along the matrix's rows
  int parts;       // of a tile's blocks of K, one a CTA or pair of a cluster
  int tiles;       // of one group of rows (of several they are counted in the kernel)
  FastDiv block_div;            // by the tiles of kBlockTiles row tiles
  FastDiv high_div[kBlockTiles + 1];  // by the row tiles of a block
  int log_box;     // of the rows of a of a copy
  int out_cols;    // columns of the output that a warp needs in its part to write them by copies
  // of a split tile (no division by the number of parts in the kernel: 100 cycles and more)
  int most;                // chunks of a part at most
  uint8_t first[9];        // the first chunk that part q joins
  uint8_t owner[16];       // the part that joins a chunk
};

struct MmSmem {
  uint32_t base;
  uint8_t* ptr;
  uint32_t bars;  // offset of two words (tensor memory's address, abort flag) and the barriers
  __device__ uint64_t* bar(int i) const { return reinterpret_cast<uint64_t*>(ptr + bars + 8) + i; }
  __device__ uint32_t* tmem_slot() const { return reinterpret_cast<uint32_t*>(ptr + bars); }
  __device__ volatile int* abort_flag() const { return reinterpret_cast<volatile int*>(ptr + bars + 4); }
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

// Two barriers, tested together: a test takes 100 cycles, most of them in flight.
__device__ __forceinline__ bool mm_warp_wait2(const MmSmem& sm, int bar0, uint32_t parity0, int bar1, uint32_t parity1,
                                              int* fault) {
  const bool a = mbar_test(smem_u32(sm.bar(bar0)), parity0), b = mbar_test(smem_u32(sm.bar(bar1)), parity1);
  if (__all_sync(0xffffffffu, a && b)) return true;
  return mm_warp_wait(sm, bar0, parity0, fault) && mm_warp_wait(sm, bar1, parity1, fault);
}

// D (+)= A B^T of 32 e4m3 of K, operands K-major with the 128-byte swizzle (8-row groups
// of 1 KB). The whole warp runs the loop around it and one elected lane issues, so the
// descriptors stay in uniform registers.
constexpr uint32_t kMmDescHigh = (1024u >> 4) | (1u << 14) | (2u << 29);  // group stride, version, swizzle
template <uint32_t kOff, int kCtas = 1>
__device__ __forceinline__ void mma_e4m3(uint32_t d, uint32_t a, uint32_t b, uint32_t idesc, uint32_t accumulate) {
  if constexpr (kCtas == 1) {
    asm volatile(
        "{\n .reg .pred p, e;\n .reg .b32 x, y;\n .reg .b64 a, b;\n add.u32 x, %1, %6;\n add.u32 y, %2, %6;\n"
        " mov.b64 a, {x, %5};\n mov.b64 b, {y, %5};\n"
        " setp.ne.b32 p, %4, 0;\n elect.sync _|e, 0xffffffff;\n"
        " @e tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], a, b, %3, p;\n}" ::"r"(d),
        "r"(a), "r"(b), "r"(idesc), "r"(accumulate), "n"(kMmDescHigh), "n"(kOff)
        : "memory");
  } else {
    asm volatile(
        "{\n .reg .pred p, e;\n .reg .b32 x, y;\n .reg .b64 a, b;\n add.u32 x, %1, %6;\n add.u32 y, %2, %6;\n"
        " mov.b64 a, {x, %5};\n mov.b64 b, {y, %5};\n"
        " setp.ne.b32 p, %4, 0;\n elect.sync _|e, 0xffffffff;\n"
        " @e tcgen05.mma.cta_group::2.kind::f8f6f4 [%0], a, b, %3, p;\n}" ::"r"(d),
        "r"(a), "r"(b), "r"(idesc), "r"(accumulate), "n"(kMmDescHigh), "n"(kOff)
        : "memory");
  }
}
__device__ __forceinline__ uint32_t mm_desc(uint32_t saddr) { return ((saddr >> 4) & 0x3FFFu) | ((16u >> 4) << 16); }

// 4 bytes to shared memory without a register.
__device__ __forceinline__ void cp_async4(uint32_t dst, const void* src) {
  asm volatile("cp.async.ca.shared.global [%0], [%1], 4;" ::"r"(dst), "l"(src) : "memory");
}
// One of the barrier's arrivals, once the thread's copies so far have landed.
__device__ __forceinline__ void cp_async_arrive(uint64_t* bar) {
  asm volatile("cp.async.mbarrier.arrive.noinc.shared::cta.b64 [%0];" ::"r"(smem_u32(bar)) : "memory");
}

__device__ __forceinline__ uint32_t cluster_rank() {
  uint32_t r;
  asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
  return r;
}
__device__ __forceinline__ uint32_t cluster_id() {
  uint32_t r;
  asm volatile("mov.u32 %0, %%clusterid.x;" : "=r"(r));
  return r;
}
__device__ __forceinline__ uint32_t clusters() {
  uint32_t r;
  asm volatile("mov.u32 %0, %%nclusterid.x;" : "=r"(r));
  return r;
}
__device__ __forceinline__ void cluster_sync() {
  asm volatile("barrier.cluster.arrive.release.aligned;\n barrier.cluster.wait.acquire.aligned;" ::: "memory");
}
// Address in CTA `rank` of the cluster of this CTA's shared address.
__device__ __forceinline__ uint32_t in_cta(uint32_t saddr, uint32_t rank) {
  uint32_t r;
  asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(r) : "r"(saddr), "r"(rank));
  return r;
}

// Registers of a warpgroup: the shares of a block add up to what it was launched with.
template <int kRegs>
__device__ __forceinline__ void mm_more_registers() {
  asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kRegs));
}
template <int kRegs>
__device__ __forceinline__ void mm_fewer_registers() {
  asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kRegs));
}

// One tile: rows row0 .. row0 + rows - 1 of a, matrix rows n0 .. of group g.
struct MmTile {
  int g, n0, row0, rows;
};

// Rows of group g, cut to what there is.
__device__ __forceinline__ void group_rows(const qsfm_matmul_params& p, int g, int& lo, int& hi, bool& bad) {
  const int a = __ldg(p.cu_rows + g), b = __ldg(p.cu_rows + g + 1);
  bad = a < 0 || b < a || b > p.rows;
  lo = min(max(a, 0), p.rows);
  hi = max(lo, min(b, p.rows));
}

// prefix[g]: tiles (of `rows` rows and one of col_tiles parts of the matrix) before group
// g's. One warp.
__device__ __forceinline__ void count_tiles(const qsfm_matmul_params& p, int rows, int col_tiles, int* prefix, int* fault) {
  const int lane = threadIdx.x & 31;
  long long run = 0;  // overlapping groups of a bad cu_rows may count more than there can be
  const auto cut = [](long long v) { return int(v < kMaxTiles ? v : kMaxTiles); };
  for (int g0 = 0; g0 < p.groups; g0 += 32) {
    long long n = 0;
    if (g0 + lane < p.groups) {
      int lo, hi;
      bool bad;
      group_rows(p, g0 + lane, lo, hi, bad);
      if (bad && blockIdx.x == 0) atomicOr(fault, QSFM_FAULT_GROUP_ROWS);
      n = (long long)((hi - lo + rows - 1) / rows) * col_tiles;
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

// Copies of a block of K into this CTA's shared memory, by one elected lane of a converged
// warp (so that what they take stays in uniform registers; a lane of its own takes 150
// cycles a copy): matrix rows, rows of a (2-D, from row y on). They complete on `bar`, of a
// pair in the first CTA.
template <int kCtas>
__device__ __forceinline__ void mm_load_w(uint32_t dst, const void* tmap, int x, int y, int z, uint32_t bar) {
  if constexpr (kCtas == 2)
    asm volatile(
        "{\n .reg .pred e;\n elect.sync _|e, 0xffffffff;\n"
        " @e cp.async.bulk.tensor.3d.cta_group::2.shared::cluster.global.mbarrier::complete_tx::bytes"
        " [%0], [%1, {%2, %3, %4}], [%5];\n}" ::"r"(dst),
        "l"(reinterpret_cast<uint64_t>(tmap)), "r"(x), "r"(y), "r"(z), "r"(bar)
        : "memory");
  else
    asm volatile(
        "{\n .reg .pred e;\n elect.sync _|e, 0xffffffff;\n"
        " @e cp.async.bulk.tensor.3d.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
        " [%0], [%1, {%2, %3, %4}], [%5];\n}" ::"r"(dst),
        "l"(reinterpret_cast<uint64_t>(tmap)), "r"(x), "r"(y), "r"(z), "r"(bar)
        : "memory");
}
template <int kCtas>
__device__ __forceinline__ void mm_load_a(uint32_t dst, const void* tmap, int x, int y, uint32_t bar) {
  if constexpr (kCtas == 2)
    asm volatile(
        "{\n .reg .pred e;\n elect.sync _|e, 0xffffffff;\n"
        " @e cp.async.bulk.tensor.2d.cta_group::2.shared::cluster.global.mbarrier::complete_tx::bytes"
        " [%0], [%1, {%2, %3}], [%4];\n}" ::"r"(dst),
        "l"(reinterpret_cast<uint64_t>(tmap)), "r"(x), "r"(y), "r"(bar)
        : "memory");
  else
    asm volatile(
        "{\n .reg .pred e;\n elect.sync _|e, 0xffffffff;\n"
        " @e cp.async.bulk.tensor.2d.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
        " [%0], [%1, {%2, %3}], [%4];\n}" ::"r"(dst),
        "l"(reinterpret_cast<uint64_t>(tmap)), "r"(x), "r"(y), "r"(bar)
        : "memory");
}
__device__ __forceinline__ void mm_expect(uint32_t bar, uint32_t bytes) {
  asm volatile(
      "{\n .reg .pred e;\n elect.sync _|e, 0xffffffff;\n"
      " @e mbarrier.arrive.expect_tx.shared::cta.b64 _, [%0], %1;\n}" ::"r"(bar), "r"(bytes)
      : "memory");
}
// Arrives on `bar` (of both CTAs of a pair, `mask`) once the MMAs issued so far have completed.
template <int kCtas>
__device__ __forceinline__ void mm_commit(uint64_t* bar, uint32_t mask) {
  if constexpr (kCtas == 2)
    asm volatile(
        "{\n .reg .pred e;\n .reg .b16 both;\n cvt.u16.u32 both, %1;\n elect.sync _|e, 0xffffffff;\n"
        " @e tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64 [%0], both;\n}"
        ::"r"(smem_u32(bar)), "r"(mask)
        : "memory");
  else
    asm volatile(
        "{\n .reg .pred e;\n elect.sync _|e, 0xffffffff;\n"
        " @e tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];\n}" ::"r"(smem_u32(bar))
        : "memory");
}
// (What it orders is tensor memory's reads, by tcgen05.fence; a release at the cluster's
// scope would wait for every load and store of the thread before it.)
__device__ __forceinline__ void arrive_in_cluster(uint32_t bar) {
  asm volatile("mbarrier.arrive.shared::cluster.b64 _, [%0];" ::"r"(bar) : "memory");
}
__device__ __forceinline__ void st_cluster(uint32_t addr, float a, float b, float c, float d) {
  asm volatile("st.shared::cluster.v4.f32 [%0], {%1, %2, %3, %4};" ::"r"(addr), "f"(a), "f"(b), "f"(c), "f"(d) : "memory");
}

__device__ __forceinline__ void prefetch_map(const CUtensorMap* map) {
  asm volatile("prefetch.tensormap [%0];" ::"l"(reinterpret_cast<uint64_t>(map)) : "memory");
}

// The walk over the tiles of a CTA or pair.
template <class C>
struct MmWalk {
  const int* prefix;
  int g, at, step, total;
  __device__ __forceinline__ bool next(const qsfm_matmul_params& p, const MmShape& s, MmTile& t) {
    constexpr int kRows = C::kRows;
    if (at >= total) return false;
    int lo = 0, hi = p.rows, local = at;
    if (p.cu_rows != nullptr) {
      while (at >= prefix[g + 1]) ++g;
      bool bad;
      group_rows(p, g, lo, hi, bad);
      local -= prefix[g];
    }
    const int row_tiles = (hi - lo + kRows - 1) / kRows;
    const int block = int(s.block_div.div(uint32_t(local)));
    const int rest = local - block * (kBlockTiles * s.col_tiles), high = min(kBlockTiles, row_tiles - block * kBlockTiles);
    const int n = int(s.high_div[high].div(uint32_t(rest))), m = block * kBlockTiles + rest - n * high;
    t.g = g;
    t.n0 = n * C::kCols;
    t.row0 = lo + m * kRows;
    t.rows = min(kRows, hi - t.row0);
    at += step;
    return true;
  }
};

// What a warp knows of its place: `cta` in the pair, the blocks b0 .. b1 - 1 of K, the
// pair's first CTA in the cluster.
struct MmPlace {
  uint32_t cta, first;
  int b0, b1;
};

// ------------------------------------------------------------- loads
template <class C>
__device__ void mm_load(const qsfm_matmul_params& p, const MmShape& s, const MmSmem& sm, MmWalk<C> walk, MmPlace at,
                        const CUtensorMap* amap, const CUtensorMap* wmap, int* fault) {
  uint32_t st = 0, par = 1;
  MmTile t;
  while (walk.next(p, s, t)) {
    // rows of a tile that are not there are not loaded, but for a pair's
    const int boxes = C::kCtas == 2 ? 1 : (t.rows + (1 << s.log_box) - 1) >> s.log_box;
    const uint32_t bytes = C::kCtas * (uint32_t(boxes << s.log_box) + C::kWRows) * kMmK;
    for (int b = at.b0; b < at.b1; ++b) {
      if (!mm_warp_wait(sm, kBEmpty + st, par, fault)) return;
      const uint32_t to = sm.base + st * C::kStage;
      const uint32_t full = smem_u32(sm.bar(kBFull + st)), bar = C::kCtas == 2 ? in_cta(full, at.first) : full;
      if (at.cta == 0) mm_expect(full, bytes);
      mm_load_w<C::kCtas>(to + C::kABytes, wmap, b * kMmK, t.n0 + int(C::kWRows * at.cta), t.g, bar);
      for (int i = 0; i < boxes; ++i)
        mm_load_a<C::kCtas>(to + (i * kMmK << s.log_box), amap, b * kMmK, t.row0 + 128 * int(at.cta) + (i << s.log_box), bar);
      if (++st == C::kStages) {
        st = 0;
        par ^= 1;
      }
    }
  }
  // the last commits' arrivals come from the pair's first CTA: the second stays until they are there
  if constexpr (C::kCtas == 2)
    for (int i = 0; i < C::kStages; ++i) {
      if (!mm_warp_wait(sm, kBEmpty + st, par, fault)) return;
      if (++st == C::kStages) {
        st = 0;
        par ^= 1;
      }
    }
}

// ------------------------------------------------------------- MMA issue
// Two warps issue in turn, `odd` the second: waiting for a stage and an accumulator and
// handing four MMAs and two commits over takes one warp 550 cycles and more, longer than
// the MMAs themselves.
template <class C>
__device__ void mm_issue(const qsfm_matmul_params& p, const MmShape& s, const MmSmem& sm, MmWalk<C> walk, MmPlace at,
                         uint32_t odd, uint32_t tmem, int* fault) {
  // formats 0 (e4m3) for both operands, as in the bf16 descriptor's f16 form
  constexpr uint32_t idesc = make_idesc_bf16(C::kRows, C::kCols, 0, 0, true);
  const uint32_t d = tmem + odd * C::kCols, mask = 3u << at.first;
  uint32_t st = odd, par = 0, tpar = 1, first = odd;  // first: whether the tile's first block is the other warp's
  MmTile t;
  while (walk.next(p, s, t)) {
    for (int b = at.b0 + int(first); b < at.b1; b += 2) {
      if (!mm_warp_wait2(sm, kBFull + st, par, kBTEmpty + odd, tpar, fault)) return;
      tc_fence_after();
      const uint32_t a = mm_desc(sm.base + st * C::kStage), w = a + (C::kABytes >> 4);
      mma_e4m3<0, C::kCtas>(d, a, w, idesc, 0);
      mma_e4m3<2, C::kCtas>(d, a, w, idesc, 1);
      mma_e4m3<4, C::kCtas>(d, a, w, idesc, 1);
      mma_e4m3<6, C::kCtas>(d, a, w, idesc, 1);
      mm_commit<C::kCtas>(sm.bar(kBTFull + odd), mask);
      mm_commit<C::kCtas>(sm.bar(kBEmpty + st), mask);
      st += 2;
      if (st >= C::kStages) {
        st = odd;
        par ^= 1;
      }
      tpar ^= 1;
    }
    first ^= uint32_t(at.b1 - at.b0) & 1;
  }
}

// ------------------------------------------------------------- scales
// Four blocks at a time, on their way to shared memory with the loads: from global
// memory, a thread's own 4 bytes a block cost the adding warps a third of their time.
template <class C>
__device__ void mm_scales(const qsfm_matmul_params& p, const MmShape& s, const MmSmem& sm, MmWalk<C> walk, MmPlace at,
                          int* fault) {
  const int lane = threadIdx.x & 31;
  uint32_t slot = 0, par = 1;
  MmTile t;
  while (walk.next(p, s, t)) {
    // rows behind the tile's take its last one's scales, and are not stored
    const int live = (min(t.rows - 128 * int(at.cta), 128) + 31) / 32;
    const float* as[4];
#pragma unroll
    for (int i = 0; i < 4; ++i)
      as[i] = p.a_scale + size_t(t.row0 + min(128 * int(at.cta) + 32 * i + lane, t.rows - 1)) * p.a_scale_row_stride +
              size_t(at.b0) * p.a_scale_col_stride;
    // lane 0 and 1: of the two halves
    const int block = min((t.n0 + C::kSums * (lane & 1)) / 128, s.col_blocks - 1);
    const float* ws = p.w_scale + (size_t(t.g) * s.col_blocks + block) * s.kb + at.b0;
    for (int b0 = at.b0; b0 < at.b1; b0 += kSlotBlocks) {
      if (!mm_warp_wait(sm, kBSEmpty + slot, par, fault)) break;
      uint32_t to = sm.base + C::kScaleAt + slot * kSlotBlocks * kSlotBlock;
      for (int b = b0; b < min(b0 + kSlotBlocks, at.b1); ++b, to += kSlotBlock) {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          if (i < live) cp_async4(to + 4 * (32 * i + lane), as[i]);
          as[i] += p.a_scale_col_stride;
        }
        if (lane < 2) cp_async4(to + 512 + 4 * lane, ws);
        ++ws;
      }
      cp_async_arrive(sm.bar(kBSFull + slot));
      if (++slot == kSlots) {
        slot = 0;
        par ^= 1;
      }
    }
  }
  asm volatile("cp.async.wait_all;" ::: "memory");
}

// ------------------------------------------------------------- sums and output
// kPart columns of the warp's 32 rows (a lane has a row) to `out`, rows `stride` elements
// apart, of which the first `rows` and `cols` are there: through shared memory (`stage`, a
// row's 16-byte pieces in turn by row), so that a warp stores whole sectors; single
// elements where the output is not aligned or ends.
template <typename T, int kPart>
__device__ __forceinline__ void store_part(T* out, size_t stride, const float* v, int rows, int cols, bool aligned,
                                           uint8_t* stage) {
  constexpr int kEach = 16 / sizeof(T), kPieces = kPart / kEach, kTurn = 8 / kPieces;
  const int lane = threadIdx.x & 31;
  const auto at = [&](int r, int piece) { return stage + 16 * kPieces * r + 16 * (piece ^ ((r / kTurn) & (kPieces - 1))); };
  __syncwarp();
#pragma unroll
  for (int i = 0; i < kPieces; ++i) {
    uint32_t w[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const int c = kEach * i + kEach / 4 * j;
      if constexpr (sizeof(T) == 4) {
        w[j] = __float_as_uint(v[c]);
      } else if constexpr (__is_same(T, __half)) {
        w[j] = pack_f16(v[c], v[c + 1]);
      } else {
        const __nv_bfloat162 h = __floats2bfloat162_rn(v[c], v[c + 1]);
        w[j] = *reinterpret_cast<const uint32_t*>(&h);
      }
    }
    *reinterpret_cast<uint4*>(at(lane, i)) = make_uint4(w[0], w[1], w[2], w[3]);
  }
  __syncwarp();
  if (aligned && kPart <= cols) {
#pragma unroll
    for (int i = 0; i < kPieces; ++i) {
      const int r = 32 / kPieces * i + lane / kPieces, piece = lane % kPieces;
      const uint4 x = *reinterpret_cast<const uint4*>(at(r, piece));
      if (r < rows) *reinterpret_cast<uint4*>(out + r * stride + piece * kEach) = x;
    }
  } else {
    for (int i = lane; i < rows * kPart; i += 32) {
      const int r = i / kPart, c = i % kPart;
      if (c < cols) out[r * stride + c] = *reinterpret_cast<const T*>(at(r, c / kEach) + c % kEach * sizeof(T));
    }
  }
}

// kN columns of the warp's rows, from element `at` of the output on.
template <int kN>
__device__ __forceinline__ void store_sums(const qsfm_matmul_params& p, size_t at, const float (&v)[kN], int rows, int cols,
                                           uint8_t* stage) {
  const int size = p.out_type == QSFM_F32 ? 4 : 2;
  const bool aligned = (reinterpret_cast<uintptr_t>(p.out) & 15) == 0 && (p.out_row_stride * size) % 16 == 0;
  constexpr int kHalf = kN < 32 ? kN : 32;  // 64 bytes of a row at a time
#pragma unroll
  for (int c = 0; c < kN; c += kHalf) {
    if (c >= cols) break;
    if (p.out_type == QSFM_BF16)
      store_part<__nv_bfloat16, kHalf>(static_cast<__nv_bfloat16*>(p.out) + at + c, p.out_row_stride, v + c, rows, cols - c,
                                       aligned, stage);
    else if (p.out_type == QSFM_F16)
      store_part<__half, kHalf>(static_cast<__half*>(p.out) + at + c, p.out_row_stride, v + c, rows, cols - c, aligned,
                                stage);
    else
#pragma unroll
      for (int h = 0; h < kHalf; h += 16)
        if (c + h < cols)
          store_part<float, 16>(static_cast<float*>(p.out) + at + c + h, p.out_row_stride, v + c + h, rows, cols - c - h,
                                aligned, stage);
  }
}

// A warp's 32 whole rows of kN columns to the output by copies, which read shared memory
// while the next tile is added up: boxes of 32 rows x 128 bytes (128-byte swizzle), two at
// a time. Columns behind the output's are not written where its rows end at 16 bytes: a copy
// writes 16 bytes at a time, whatever of them lies within the map.
template <typename T, int kN>
__device__ __forceinline__ void store_boxes(const CUtensorMap* omap, const float (&v)[kN], int row, int n0, int n,
                                            uint32_t stage) {
  constexpr int kBox = 128 / sizeof(T), kEach = 16 / sizeof(T);
  const int lane = threadIdx.x & 31;
#pragma unroll
  for (int c0 = 0; c0 < kN; c0 += 2 * kBox) {
    if (n0 + c0 >= n) break;
    if (lane == 0) asm volatile("cp.async.bulk.wait_group.read 0;" ::: "memory");  // the last boxes have been read
    __syncwarp();
#pragma unroll
    for (int h = 0; h < 2 * kBox && c0 + h < kN; h += kBox) {
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        uint32_t w[4];
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const int c = c0 + h + kEach * i + kEach / 4 * j;
          if constexpr (sizeof(T) == 4) {
            w[j] = __float_as_uint(v[c]);
          } else if constexpr (__is_same(T, __half)) {
            w[j] = pack_f16(v[c], v[c + 1]);
          } else {
            const __nv_bfloat162 x = __floats2bfloat162_rn(v[c], v[c + 1]);
            w[j] = *reinterpret_cast<const uint32_t*>(&x);
          }
        }
        sts_v4(stage + (h / kBox) * kOutBox + 128 * lane + 16 * (i ^ (lane & 7)), make_uint4(w[0], w[1], w[2], w[3]));
      }
    }
    fence_proxy_async_smem();
    __syncwarp();
    if (lane == 0) {
#pragma unroll
      for (int h = 0; h < 2 * kBox && c0 + h < kN; h += kBox)
        if (n0 + c0 + h < n)
          asm volatile("cp.async.bulk.tensor.2d.global.shared::cta.bulk_group [%0, {%1, %2}], [%3];" ::"l"(
                           reinterpret_cast<uint64_t>(omap)),
                       "r"(n0 + c0 + h), "r"(row), "r"(stage + (h / kBox) * kOutBox)
                       : "memory");
      asm volatile("cp.async.bulk.commit_group;" ::: "memory");
    }
  }
}

// Adds up a tile's blocks; false after a timeout. Warps without rows (kLive false) keep
// step with the others.
template <class C, bool kLive>
__device__ __forceinline__ bool mm_add(const MmShape& s, const MmSmem& sm, MmPlace at, uint32_t tmem, uint32_t tempty,
                                       uint32_t& buf, uint32_t& tpar, uint32_t& slot, uint32_t& spar,
                                       float (&acc)[C::kSums], int* fault) {
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, half = warp >> 2;
  if constexpr (kLive) {
#pragma unroll
    for (int i = 0; i < C::kSums; ++i) acc[i] = 0.f;
  }
  for (int b0 = at.b0; b0 < at.b1; b0 += kSlotBlocks) {
    if (!mm_warp_wait(sm, kBSFull + slot, spar, fault)) return false;
    const float* scales = reinterpret_cast<const float*>(sm.ptr + C::kScaleAt + slot * kSlotBlocks * kSlotBlock);
    for (int b = b0; b < min(b0 + kSlotBlocks, at.b1); ++b, scales += kSlotBlock / 4) {
      const float f = kLive ? scales[32 * (warp & 3) + lane] * scales[128 + half] : 0.f;
      if (!mm_warp_wait(sm, kBTFull + buf, tpar, fault)) return false;
      tc_fence_after();
      const uint32_t from = tmem + buf * C::kCols + C::kSums * half + (uint32_t(32 * (warp & 3)) << 16);
#pragma unroll
      for (int c = 0; c < C::kSums; c += C::kRound) {
        float v[C::kRound];
        if constexpr (kLive) {
#pragma unroll
          for (int j = 0; j < C::kRound; j += 32) tmem_ld32(from + c + j, v + j);
          tmem_ld_wait();
        }
        if (c + C::kRound >= C::kSums) {  // the accumulator is free as soon as the last round has it
          tc_fence_before();
          __syncwarp();
          if (lane == 0) {
            if constexpr (C::kCtas == 2) arrive_in_cluster(tempty + 8 * buf);
            else mbar_arrive(sm.bar(kBTEmpty + buf));
          }
        }
        if constexpr (kLive) {
#pragma unroll
          for (int j = 0; j < C::kRound; ++j) acc[c + j] = fmaf(v[j], f, acc[c + j]);
        }
      }
      buf ^= 1;
      tpar ^= buf == 0;
    }
    __syncwarp();
    if (lane == 0) mbar_arrive(sm.bar(kBSEmpty + slot));
    if (++slot == kSlots) {
      slot = 0;
      spar ^= 1;
    }
  }
  return true;
}

template <class C>
__device__ void mm_sum(const qsfm_matmul_params& p, const MmShape& s, const MmSmem& sm, MmWalk<C> walk, MmPlace at,
                       uint32_t tmem, const CUtensorMap* omap, int* fault) {
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int row0 = 128 * int(at.cta) + 32 * (warp & 3), half = warp >> 2;
  const uint32_t tempty = in_cta(smem_u32(sm.bar(kBTEmpty)), at.first);
  uint8_t* stage = sm.ptr + (s.parts == 1 ? C::kOutAt + C::kOutWarp * warp : C::kJoinedAt + kOutPart * warp);
  uint32_t buf = 0, tpar = 0, slot = 0, spar = 0;
  MmTile t;
  float acc[C::kSums];
  if (s.parts == 1) {
    while (walk.next(p, s, t)) {
      const int rows = min(32, t.rows - row0), n0 = t.n0 + C::kSums * half, cols = p.n - n0;
      if (rows <= 0) {
        if (!mm_add<C, false>(s, sm, at, tmem, tempty, buf, tpar, slot, spar, acc, fault)) return;
        continue;
      }
      if (!mm_add<C, true>(s, sm, at, tmem, tempty, buf, tpar, slot, spar, acc, fault)) return;
      if (cols <= 0) continue;
      if (C::kBoxes && cols >= s.out_cols && rows == 32) {
        const uint32_t boxes = sm.base + C::kOutAt + C::kOutWarp * warp;
        if (p.out_type == QSFM_BF16) store_boxes<__nv_bfloat16>(omap, acc, t.row0 + row0, n0, p.n, boxes);
        else if (p.out_type == QSFM_F16) store_boxes<__half>(omap, acc, t.row0 + row0, n0, p.n, boxes);
        else store_boxes<float>(omap, acc, t.row0 + row0, n0, p.n, boxes);
      } else {
        if (C::kBoxes && lane == 0) asm volatile("cp.async.bulk.wait_group.read 0;" ::: "memory");
        store_sums(p, size_t(t.row0 + row0) * p.out_row_stride + n0, acc, rows, cols, stage);
      }
    }
    if (C::kBoxes && lane == 0) asm volatile("cp.async.bulk.wait_group 0;" ::: "memory");
    return;
  }
  // The cluster's one tile: its part q adds up the chunks n q / parts .. of the tile's n
  // chunks of 16 columns, in the order of the parts. The sums take the place of the
  // operands, which every CTA of the cluster is through with at the first barrier: of part
  // q's chunk c from part r at [r][c - first of q][4][128 rows][4 columns].
  bool ok = walk.next(p, s, t);
  const int rows = ok ? min(32, t.rows - row0) : 0;
  if (ok)
    ok = rows > 0 ? mm_add<C, true>(s, sm, at, tmem, tempty, buf, tpar, slot, spar, acc, fault)
                  : mm_add<C, false>(s, sm, at, tmem, tempty, buf, tpar, slot, spar, acc, fault);
  const int part = int(at.first) / C::kCtas;
  cluster_sync();
  if (ok && lane < rows) {
#pragma unroll
    for (int c = 0; c < C::kSums; c += kChunk) {
      const int chunk = (C::kSums * half + c) / kChunk;
      const int owner = s.owner[chunk], place = part * s.most + chunk - s.first[owner];
      const uint32_t to = in_cta(sm.base + place * kChunkBytes + 16 * ((row0 & 127) + lane), uint32_t(owner * C::kCtas) + at.cta);
#pragma unroll
      for (int i = 0; i < kChunk; i += 4) st_cluster(to + 512 * i, acc[c + i], acc[c + i + 1], acc[c + i + 2], acc[c + i + 3]);
    }
  }
  cluster_sync();
  if (!ok || rows <= 0) return;
  const uint8_t* sums = sm.ptr + 16 * ((row0 & 127) + lane);
  const int c0 = s.first[part], c1 = s.first[part + 1];
  for (int c = c0 + half; c < c1; c += 2) {
    const int n0 = t.n0 + kChunk * c;
    if (n0 >= p.n) break;
    float v[kChunk];
    for (int q = 0; q < s.parts; ++q) {
      const uint8_t* from = sums + (q * s.most + c - c0) * kChunkBytes;
#pragma unroll
      for (int i = 0; i < kChunk; i += 4) {
        const float4 x = *reinterpret_cast<const float4*>(from + 512 * i);
        v[i] = q == 0 ? x.x : v[i] + x.x;
        v[i + 1] = q == 0 ? x.y : v[i + 1] + x.y;
        v[i + 2] = q == 0 ? x.z : v[i + 2] + x.z;
        v[i + 3] = q == 0 ? x.w : v[i + 3] + x.w;
      }
    }
    store_sums(p, size_t(t.row0 + row0) * p.out_row_stride + n0, v, rows, p.n - n0, stage);
  }
}

// ------------------------------------------------------------- the kernel
template <class C>
__global__ void __launch_bounds__(kMmThreads, 1)
    matmul_kernel(const __grid_constant__ qsfm_matmul_params p, const __grid_constant__ MmShape s, int* fault,
                  const __grid_constant__ CUtensorMap amap, const __grid_constant__ CUtensorMap wmap,
                  const __grid_constant__ CUtensorMap omap) {
  extern __shared__ uint8_t mm_smem[];
  const uint32_t raw = smem_u32(mm_smem);
  MmSmem sm;
  sm.base = (raw + 1023u) & ~1023u;
  sm.ptr = mm_smem + (sm.base - raw);
  sm.bars = C::kBarAt;
  const int tid = threadIdx.x, warp = tid >> 5;
  const bool cluster = C::kCtas == 2 || s.parts > 1;
  const uint32_t rank = cluster ? cluster_rank() : 0;
  int* prefix = reinterpret_cast<int*>(sm.ptr + C::kPrefixAt);
  if (tid < kBCount) {  // a barrier each
    const int i = tid;
    mbar_init(sm.bar(i), i >= kBTEmpty && i < kBDrain     ? C::kCtas * kAddWarps
                         : i >= kBSFull && i < kBSEmpty ? 32
                         : i >= kBSEmpty                ? kAddWarps
                                                        : 1);
    if (tid == 0) *sm.abort_flag() = 0;
    fence_mbar_init();
  }
  if (warp == kAddWarps && (tid & 31) == 0) {
    prefetch_map(&amap);
    prefetch_map(&wmap);
  }
  if (warp == kAddWarps + 1) {  // of both CTAs
    if constexpr (C::kCtas == 2) {
      asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_u32(sm.tmem_slot())),
                   "r"(C::kTmem)
                   : "memory");
      asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;" ::: "memory");
    } else {
      tmem_alloc(sm.tmem_slot(), C::kTmem);
    }
  }
  grid_dependency_wait();
  grid_launch_dependents();
  if (warp == 0 && p.cu_rows != nullptr) count_tiles(p, C::kRows, s.col_tiles, prefix, fault);
  tc_fence_before();
  __syncthreads();
  if (cluster) cluster_sync();  // barriers and tensor memory of all CTAs are there
  tc_fence_after();
  const uint32_t tmem = *sm.tmem_slot();
  MmPlace at;
  at.cta = rank & (C::kCtas - 1);
  at.first = rank - at.cta;
  const int part = int(at.first) / C::kCtas;
  at.b0 = s.parts == 1 ? 0 : int(uint32_t(s.kb * part) / uint32_t(s.parts));
  at.b1 = s.parts == 1 ? s.kb : int(uint32_t(s.kb * (part + 1)) / uint32_t(s.parts));
  MmWalk<C> walk;
  walk.prefix = prefix;
  walk.g = 0;
  walk.at = int(cluster_id());
  walk.step = int(clusters());
  walk.total = p.cu_rows != nullptr ? prefix[p.groups] : s.tiles;
  if (warp < kAddWarps) {
    mm_more_registers<kAddRegs>();
    mm_sum<C>(p, s, sm, walk, at, tmem, &omap, fault);
  } else {
    mm_fewer_registers<kOtherRegs>();
    if (warp == kAddWarps) {
      mm_load<C>(p, s, sm, walk, at, &amap, &wmap, fault);
    } else if (warp == kAddWarps + 3) {
      mm_scales<C>(p, s, sm, walk, at, fault);
    } else if (at.cta == 0) {
      const int odd = warp - kAddWarps - 1;
      mm_issue<C>(p, s, sm, walk, at, uint32_t(odd), tmem, fault);
      // every MMA issued has completed before tensor memory is freed
      mm_commit<C::kCtas>(sm.bar(kBDrain + odd), 1u << at.first);
      volatile int never = 0;
      if (!mbar_wait_poll(smem_u32(sm.bar(kBDrain + odd)), 0, &never, kMmTimeoutNs)) atomicOr(fault, QSFM_FAULT_TIMEOUT);
    }
    __syncwarp();
    if (s.parts > 1) {  // (the adding warps' are in mm_sum)
      cluster_sync();
      cluster_sync();
    }
  }
  // after an abort copies may still be on their way into this CTA's shared memory:
  // a millisecond is far more than they take
  if (warp == kAddWarps && *sm.abort_flag())
    for (int i = 0; i < 1000; ++i) __nanosleep(1000);
  __syncwarp();
  tc_fence_before();
  __syncthreads();
  // the other CTA's accumulators are read, its arrivals are there (the commits': mm_load's last waits)
  if (C::kCtas == 2) cluster_sync();
  if (warp == kAddWarps + 1) {
    tc_fence_after();
    if constexpr (C::kCtas == 2)
      asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(C::kTmem) : "memory");
    else
      tmem_dealloc(tmem, C::kTmem);
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

// A tensor map by `call`. The encoder is a driver call and wants a context, which a host
// thread has from its first runtime call that needs one: the product may be that thread's
// first (what it asks of the device before is answered without), so it is bound here.
template <class Call>
cudaError_t encode_map(const Call& call) {
  CUresult r = call();
  if (r == CUDA_ERROR_INVALID_CONTEXT || r == CUDA_ERROR_NOT_INITIALIZED) {
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e == cudaSuccess) e = cudaSetDevice(dev);
    if (e != cudaSuccess) return e;
    r = call();
  }
  return r == CUDA_SUCCESS ? cudaSuccess : cudaErrorInvalidValue;
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
  return encode_map([&] {
    return encode(map, CU_TENSOR_MAP_DATA_TYPE_UINT8, is3d ? 3 : 2, const_cast<void*>(base), dims, strides, box, estr,
                  CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                  CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
  });
}

// The output in boxes of 32 rows x 128 bytes.
cudaError_t make_out_map(const qsfm_matmul_params& p, int size, CUtensorMap* map) {
  const auto encode = tensor_map_encoder();
  if (encode == nullptr) return cudaErrorNotSupported;
  const long long stride = p.rows == 1 ? (p.n * (long long)size + 15) & ~15ll : p.out_row_stride * size;
  const cuuint64_t dims[2] = {cuuint64_t(p.n), cuuint64_t(p.rows)}, strides[1] = {cuuint64_t(stride)};
  const cuuint32_t box[2] = {cuuint32_t(128 / size), 32}, estr[2] = {1, 1};
  const CUtensorMapDataType type = p.out_type == QSFM_F32   ? CU_TENSOR_MAP_DATA_TYPE_FLOAT32
                                   : p.out_type == QSFM_F16 ? CU_TENSOR_MAP_DATA_TYPE_FLOAT16
                                                            : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16;
  return encode_map([&] {
    return encode(map, type, 2, p.out, dims, strides, box, estr, CU_TENSOR_MAP_INTERLEAVE_NONE,
                  CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_NONE, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
  });
}

constexpr int kMaxDevices = 64;

// Prepares a device for a kernel, once: its shared memory, and that it has the registers
// that the split counts on (with fewer the adding warps would wait forever).
template <class C>
cudaError_t prepare(int dev) {
  static std::atomic<bool> done[kMaxDevices];
  if (dev < kMaxDevices && done[dev].load(std::memory_order_relaxed)) return cudaSuccess;
  cudaFuncAttributes attr;
  cudaError_t e = cudaFuncGetAttributes(&attr, matmul_kernel<C>);
  if (e != cudaSuccess) return e;
  if (attr.numRegs < kLaunchRegs) return cudaErrorInvalidConfiguration;
  e = cudaFuncSetAttribute(matmul_kernel<C>, cudaFuncAttributeMaxDynamicSharedMemorySize, int(C::kSmem));
  if (e == cudaSuccess && dev < kMaxDevices) done[dev].store(true, std::memory_order_relaxed);
  return e;
}

// Clusters of `size` CTAs that run at a time, 0 if none: fewer than SMs / size, since each
// lies in one part of the GPU (36 of four, 23 of six, 15 of eight on 152 SMs). Looked up
// once for a device.
template <class C>
int active_clusters(int dev, int sms, int size) {
  if (size == 1) return sms;
  static std::atomic<int> known[kMaxDevices][9];
  int n = dev < kMaxDevices ? known[dev][size].load(std::memory_order_relaxed) : 0;
  if (n == 0) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(unsigned(size * sms));
    cfg.blockDim = dim3(kMmThreads);
    cfg.dynamicSmemBytes = C::kSmem;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = unsigned(size);
    attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    if (cudaOccupancyMaxActiveClusters(&n, matmul_kernel<C>, &cfg) != cudaSuccess || n < 1) n = -1;
    if (dev < kMaxDevices) known[dev][size].store(n, std::memory_order_relaxed);
  }
  return n > 0 ? n : 0;
}

// How long a product takes with tiles of C, in microseconds, as fitted to 16 shapes of 1 to
// 4096 rows, 1000 to 32768 matrix rows and K of 1024 to 32768 with every number of parts
// (the shortest of them within 10% of the estimate's choice): a launch, per round of tiles
// the blocks of K and what a tile takes besides, or the matrices' bytes at the rate that
// they arrive at, and the join of a split tile, which grows with its rows.
struct MmTimes {
  double block, tile, join, join_rows;
};
constexpr MmTimes kPairTimes = {0.41, 1.9, 2.0, 3.5}, kWideTimes = {0.43, 2.2, 2.0, 3.5}, kSmallTimes = {0.36, 1.0, 1.5, 2.0};
constexpr double kLaunchTime = 2.5, kBytesPerUs = 6.2e6;

struct MmPlan {
  long long tiles;  // at most
  int parts;        // of a tile's blocks of K
  double time;
};

// The tiles of one group are known here, and where they leave SMs without work they are
// split; of several groups the tiles are a guess, and not split.
template <class C>
MmPlan plan(const qsfm_matmul_params& p, int dev, int sms, const MmTimes& times) {
  const int kb = (p.k + kMmK - 1) / kMmK;
  const long long col_tiles = (p.n + C::kCols - 1) / C::kCols;
  MmPlan best = {0, 1, 0};
  double tiles, rows, groups = 1;
  if (p.cu_rows == nullptr) {
    best.tiles = (long long)((p.rows + C::kRows - 1) / C::kRows) * col_tiles;
    rows = p.rows;
    tiles = double(best.tiles);
  } else {
    // every group but one may add a tile that is not full
    groups = p.groups < p.rows ? p.groups : p.rows;
    best.tiles = ((long long)p.rows / C::kRows + (long long)groups) * col_tiles;
    rows = p.rows / groups;
    tiles = groups * (rows <= C::kRows / 2 ? 1 : rows / C::kRows + 0.5) * col_tiles;
  }
  const double bytes = (groups * p.n + p.rows) * p.k / kBytesPerUs;
  for (int parts = 1; parts * C::kCtas <= 8 && (parts == 1 || 2 * parts <= kb); ++parts) {
    const long long room = active_clusters<C>(dev, sms, parts * C::kCtas);
    if (parts > 1 && (p.cu_rows != nullptr || best.tiles > room)) continue;  // split tiles all run at once
    const double rounds = std::ceil(tiles / double(room > 0 ? room : 1));
    const double work = rounds * ((kb + parts - 1) / parts * times.block + times.tile);
    const double time = kLaunchTime + (work > bytes ? work : bytes) +
                        (parts > 1 ? times.join + times.join_rows * (rows < 128 ? rows : 128) / 128 : 0);
    if (parts == 1 || time < best.time) {
      best.parts = parts;
      best.time = time;
    }
  }
  return best;
}

template <class C>
cudaError_t launch_ctas(const qsfm_matmul_params& p, const MmPlan& plan, int rows, int sms, int* fault,
                        cudaStream_t stream) {
  cudaError_t e;
  MmShape s;
  s.kb = (p.k + kMmK - 1) / kMmK;
  s.col_blocks = (p.n + 127) / 128;
  s.col_tiles = (p.n + C::kCols - 1) / C::kCols;
  s.parts = plan.parts;
  s.tiles = int(plan.tiles);
  s.block_div.set(uint32_t(kBlockTiles * s.col_tiles));
  for (int i = 1; i <= kBlockTiles; ++i) s.high_div[i].set(uint32_t(i));
  // as many rows of a as a tile has (a copy takes its time to issue), few where it has few
  s.log_box = C::kCtas == 2 || rows > 64 ? 7 : rows > 32 ? 6 : 5;
  constexpr int kChunks = C::kCols / kChunk;
  s.most = (kChunks + s.parts - 1) / s.parts;
  for (int q = 0; q <= s.parts; ++q) s.first[q] = uint8_t(kChunks * q / s.parts);
  for (int q = 0; q < s.parts; ++q)
    for (int c = s.first[q]; c < s.first[q + 1]; ++c) s.owner[c] = uint8_t(q);
  CUtensorMap amap, wmap;
  if ((e = make_map(p.a, p.k, p.rows, 1, p.a_row_stride, 0, 1 << s.log_box, false, &amap)) != cudaSuccess)
    return e;
  if ((e = make_map(p.w, p.k, p.n, p.groups, p.w_row_stride, p.w_group_stride, int(C::kWRows), true, &wmap)) != cudaSuccess)
    return e;
  CUtensorMap omap = amap;  // (not used)
  const int size = p.out_type == QSFM_F32 ? 4 : 2;
  const bool boxes = C::kBoxes && s.parts == 1 && (reinterpret_cast<uintptr_t>(p.out) & 15) == 0 &&
                     (p.rows == 1 || (p.out_row_stride * size) % 16 == 0);
  s.out_cols = !boxes ? INT_MAX : (p.n * (long long)size) % 16 == 0 ? 1 : C::kSums;
  if (boxes && (e = make_out_map(p, size, &omap)) != cudaSuccess) return e;
  const long long room = sms / C::kCtas;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(unsigned(C::kCtas * (s.parts > 1 ? plan.tiles * s.parts : plan.tiles < room ? plan.tiles : room)));
  cfg.blockDim = dim3(kMmThreads);
  cfg.dynamicSmemBytes = C::kSmem;
  cfg.stream = stream;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = unsigned(C::kCtas * s.parts);
  attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = C::kCtas * s.parts > 1 ? 2 : 1;
  return cudaLaunchKernelEx(&cfg, matmul_kernel<C>, p, s, fault, amap, wmap, omap);
}

using Pair = Mm<2, 256>;
using Wide = Mm<1, 256>;
using Small = Mm<1, 128>;

// The kernel of a product, prepared on the current device, and its parts.
struct MmChoice {
  int ctas, cols;  // of its tiles
  int sms;
  MmPlan plan;
};

cudaError_t choose(const qsfm_matmul_params& p, MmChoice& c) {
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  if ((e = cudaDeviceGetAttribute(&c.sms, cudaDevAttrMultiProcessorCount, dev)) != cudaSuccess) return e;
  if ((e = prepare<Pair>(dev)) != cudaSuccess || (e = prepare<Wide>(dev)) != cudaSuccess ||
      (e = prepare<Small>(dev)) != cudaSuccess)
    return e;
  const MmPlan pair = plan<Pair>(p, dev, c.sms, kPairTimes), wide = plan<Wide>(p, dev, c.sms, kWideTimes),
               small = plan<Small>(p, dev, c.sms, kSmallTimes);
  // (the pair first where it is as good: it reads a third less)
  const bool paired = pair.time <= 1.03 * wide.time && pair.time <= 1.03 * small.time;
  c.plan = paired ? pair : wide.time <= small.time ? wide : small;
  c.ctas = paired ? Pair::kCtas : 1;
  c.cols = paired || wide.time <= small.time ? Wide::kCols : Small::kCols;
  return cudaSuccess;
}

}  // namespace

cudaError_t launch_matmul(const qsfm_matmul_params& p, int* fault, cudaStream_t stream) {
  MmChoice c;
  const cudaError_t e = choose(p, c);
  if (e != cudaSuccess) return e;
  const int rows = (p.rows + p.groups - 1) / p.groups;  // of a group, on average
  if (c.ctas == Pair::kCtas) return launch_ctas<Pair>(p, c.plan, rows, c.sms, fault, stream);
  return c.cols == Wide::kCols ? launch_ctas<Wide>(p, c.plan, rows, c.sms, fault, stream)
                               : launch_ctas<Small>(p, c.plan, rows, c.sms, fault, stream);
}

cudaError_t matmul_plan(const qsfm_matmul_params& p, int32_t* rows, int32_t* columns, int32_t* parts) {
  MmChoice c;
  const cudaError_t e = choose(p, c);
  if (e != cudaSuccess) return e;
  *rows = 128 * c.ctas;
  *columns = c.cols;
  *parts = c.plan.parts;
  return cudaSuccess;
}

}  // namespace qsfm
