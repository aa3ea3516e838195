// Parts the attention kernels share: the walk over a CTA's planned pieces,
// bounded waits, lane reductions, the tensor map of q.
//
// A kernel's shared-memory view (the template argument Smem) offers bar(i) and
// abort_flag().
#pragma once

#include <cuda.h>
#include <cudaTypedefs.h>
#include <cuda_runtime.h>

#include <mutex>

#include "qsfm_device.cuh"
#include "qsfm_internal.h"

namespace qsfm {
namespace {

constexpr float kRescaleLog2 = 8.0f;
constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.6931471805599453f;
constexpr uint64_t kTimeoutNs = 2000000000ull;  // 2 s per wait

struct Range {
  int t0, k0, t1, k1;
};

// Walks the (unit, tile-range) pieces of a CTA's range in order.
struct PieceIter {
  const qsfm_params* p;
  Range r;
  int T;
  int t;
  __device__ PieceIter(const qsfm_params* p_, Range r_, int T_) : p(p_), r(r_), T(T_), t(r_.t0) {}
  __device__ bool next(int& tok, TokenGeom& g, int& lo, int& hi) {
    if (t > r.t1 || t >= T || (t == r.t1 && r.k1 == 0)) return false;
    tok = t;
    g = token_geom(*p, t);
    lo = (t == r.t0) ? min(r.k0, g.n_tiles) : 0;
    hi = (t == r.t1) ? min(r.k1, g.n_tiles) : g.n_tiles;
    ++t;
    return true;
  }
};

__device__ __forceinline__ uint32_t pack_bf16(float a, float b) {
  __nv_bfloat162 v = __floats2bfloat162_rn(a, b);
  return *reinterpret_cast<uint32_t*>(&v);
}

// Max (kMax) or sum of kN (16 or 32) values per lane over the 32 lanes of a
// warp, by halving exchanges (for kN = 16, lanes l and l ^ 16 are combined
// first): afterwards lane l holds the result for value index l % kN. The
// array is consumed.
template <bool kMax, int kN>
__device__ __forceinline__ float reduce_lanes(float (&v)[kN]) {
  const int lane = threadIdx.x & 31;
  if constexpr (kN == 16) {
#pragma unroll
    for (int i = 0; i < 16; ++i) {
      const float got = __shfl_xor_sync(0xffffffffu, v[i], 16);
      v[i] = kMax ? fmaxf(v[i], got) : v[i] + got;
    }
  }
#pragma unroll
  for (int w = kN / 2; w >= 1; w >>= 1) {
    const bool up = lane & w;
#pragma unroll
    for (int i = 0; i < w; ++i) {
      const float keep = up ? v[w + i] : v[i];
      const float send = up ? v[i] : v[w + i];
      const float got = __shfl_xor_sync(0xffffffffu, send, w);
      v[i] = kMax ? fmaxf(keep, got) : keep + got;
    }
  }
  return v[0];
}

// kN consecutive tensor-memory columns of the warp's 32 lanes, one lane per
// thread.
template <int kN>
__device__ __forceinline__ void tmem_load(uint32_t taddr, float (&v)[kN]) {
  if constexpr (kN == 32) tmem_ld32(taddr, v);
  else tmem_ld16(taddr, v);
}
template <int kN>
__device__ __forceinline__ void tmem_store(uint32_t taddr, const float (&v)[kN]) {
  if constexpr (kN == 32) tmem_st32(taddr, v);
  else tmem_st16(taddr, v);
}

// Bounded wait; on timeout raises the CTA's abort flag and the fault bit.
template <typename Smem>
__device__ __forceinline__ bool wait_or_abort(const Smem& sm, int bar, uint32_t parity, int* fault) {
  if (mbar_wait_bounded(sm.bar(bar), parity, sm.abort_flag(), kTimeoutNs)) return true;
  if (!*sm.abort_flag()) {
    *sm.abort_flag() = 1;
    atomicOr(fault, QSFM_FAULT_TIMEOUT);
  }
  return false;
}

// Warp-uniform bounded wait: lane 0 polls, the result is broadcast, so the
// lanes of a warp never split on a timeout.
template <typename Smem>
__device__ __forceinline__ bool warp_wait_or_abort(const Smem& sm, int bar, uint32_t parity,
                                                   int* fault) {
  bool ok = true;
  if ((threadIdx.x & 31) == 0) ok = wait_or_abort(sm, bar, parity, fault);
  __syncwarp();  // the other lanes wait here (and are ordered after lane 0's acquire)
  return __shfl_sync(0xffffffffu, ok ? 1 : 0, 0) != 0;
}

__device__ __forceinline__ float e8m0_value(uint32_t e) {
  // 2^(e - 127): the fp32 with biased exponent e (e = 0: the subnormal 2^-127)
  return e == 0xFFu ? __uint_as_float(0x7FC00000u) : e == 0u ? __uint_as_float(0x00400000u)
                                                             : __uint_as_float(e << 23);
}

// Runs before the plan is readable, while the plan kernel still runs: warms
// L2 with the Q and the sparse-index row of the unit this CTA most likely
// starts with (the plan cuts equal-cost units evenly, so CTA c of G starts
// near unit c T / G). Prefetches only, no loads to wait for, no fault bits:
// a wrong guess costs bandwidth, never results or time.
__device__ __forceinline__ void warm_first_token(const qsfm_params& p, int T, int c, int G, int lane) {
  const int t = int((long long)c * T / G);
  if (t >= T) return;
  if (lane == 0)
    bulk_prefetch_l2(static_cast<const uint8_t*>(p.q) + size_t(t) * kHeads * kDim * 2, kHeads * kDim * 2);
  if (p.cmp_sparse_indices != nullptr) {
    const uint8_t* ix = reinterpret_cast<const uint8_t*>(p.cmp_sparse_indices + size_t(t >> unit_shift(p)) * p.k2);
    for (int off = 128 * lane; off < 4 * p.k2; off += 32 * 128) prefetch_l2(ix + off);
  }
}

// Tensor map of q viewed as [T * 64 rows, 512 bf16 columns], boxes of 64 rows
// (the heads of a unit) x 64 columns (128 B) with the 128-B swizzle of the MMA
// operand.
cudaError_t make_q_map(const void* q, int T, CUtensorMap* map) {
  static PFN_cuTensorMapEncodeTiled_v12000 encode = nullptr;
  static std::once_flag once;
  std::call_once(once, [] {
    cudaDriverEntryPointQueryResult qres;
    void* fn = nullptr;
    if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &fn, 12000, cudaEnableDefault,
                                         &qres) == cudaSuccess &&
        qres == cudaDriverEntryPointSuccess)
      encode = reinterpret_cast<PFN_cuTensorMapEncodeTiled_v12000>(fn);
  });
  if (encode == nullptr) return cudaErrorNotSupported;
  const cuuint64_t dims[2] = {cuuint64_t(kDim), cuuint64_t(T) * kHeads};
  const cuuint64_t strides[1] = {cuuint64_t(kDim) * 2};
  const cuuint32_t box[2] = {64, 64};
  const cuuint32_t estr[2] = {1, 1};
  const CUresult r = encode(map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 2, const_cast<void*>(q), dims,
                            strides, box, estr, CU_TENSOR_MAP_INTERLEAVE_NONE,
                            CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_128B,
                            CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
  return r == CUDA_SUCCESS ? cudaSuccess : cudaErrorInvalidValue;
}

}  // namespace
}  // namespace qsfm
