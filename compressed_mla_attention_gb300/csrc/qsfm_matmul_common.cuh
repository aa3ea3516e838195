// Shared by the two kernels of the 8-bit products: barriers, copies, MMAs, the walk over
// tiles and the tensor maps.
#pragma once

#include <cuda.h>
#include <cudaTypedefs.h>
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include <mutex>

#include "qsfm_device.cuh"
#include "qsfm_internal.h"

namespace qsfm {

constexpr int kMmK = 128;            // bytes of K per stage: one block of scales
constexpr int kMmMaxGroups = 1024;
constexpr long long kMmMaxTiles = (1ll << 30) + 1;  // counted at most
constexpr uint64_t kMmTimeoutNs = 1000000000ull;
constexpr uint32_t kMmSmemMax = 227 * 1024;

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

__device__ __forceinline__ void mm_load_3d(uint32_t dst, const void* tmap, int x, int y, int z, uint64_t* bar) {
  asm volatile(
      "cp.async.bulk.tensor.3d.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
      " [%0], [%1, {%2, %3, %4}], [%5];" ::"r"(dst),
      "l"(reinterpret_cast<uint64_t>(tmap)), "r"(x), "r"(y), "r"(z), "r"(smem_u32(bar))
      : "memory");
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

// 4 bytes to shared memory without a register, zeros where `bytes` is 0.
__device__ __forceinline__ void cp_async4(uint32_t dst, const void* src, uint32_t bytes) {
  asm volatile("cp.async.ca.shared.global [%0], [%1], 4, %2;" ::"r"(dst), "l"(src), "r"(bytes) : "memory");
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

// prefix[g]: tiles (of `rows` rows and one of col_tiles parts of the matrix) before group
// g's. One warp.
__device__ __forceinline__ void count_tiles(const qsfm_matmul_params& p, int rows, int col_tiles, int* prefix, int* fault) {
  const int lane = threadIdx.x & 31;
  long long run = 0;  // overlapping groups of a bad cu_rows may count more than there can be
  const auto cut = [](long long v) { return int(v < kMmMaxTiles ? v : kMmMaxTiles); };
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

__device__ __forceinline__ void mm_store(const qsfm_matmul_params& p, size_t at, float v) {
  if (p.out_type == QSFM_BF16) static_cast<__nv_bfloat16*>(p.out)[at] = __float2bfloat16(v);
  else if (p.out_type == QSFM_F16) static_cast<__half*>(p.out)[at] = __float2half(v);
  else static_cast<float*>(p.out)[at] = v;
}

// ------------------------------------------------------------- host side
inline PFN_cuTensorMapEncodeTiled_v12000 mm_tensor_map_encoder() {
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
inline cudaError_t make_map(const void* base, int k, int rows, int planes, long long row_stride, long long plane_stride,
                     int box_rows, bool is3d, CUtensorMap* map) {
  const auto encode = mm_tensor_map_encoder();
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

// The kernel of many rows (qsfm_matmul_pair.cu).
cudaError_t launch_matmul_pair(const qsfm_matmul_params& p, int sms, int* fault, cudaStream_t stream);

}  // namespace qsfm
