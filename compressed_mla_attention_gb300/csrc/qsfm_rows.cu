// Norm, position rotation and cache store of query and key rows (sm_103a).
//
// For each head row x of a token (512 elements):
//   y = x / sqrt(mean(x^2) + eps) * weight, then the rope_dim elements from
//   rope_offset on are turned by the token's angles,
// rounded once: queries to bf16, the token's one latent key row to its cache
// row format (bf16, e4m3 with fp32 or e8m0 scales, e2m1 with e4m3 scales).
//
// One warp per row: lane l holds elements 8 l .. + 7 of each 256-element half
// (two 16-byte loads of a bf16 row), so the sum of squares is five shuffles,
// the pairs of a rotation are in the lane (adjacent) or rope_dim / 16 lanes
// apart (halves), and a quantisation group of 16 or 64 elements is 2 or 8
// neighbouring lanes. A row is read once, held in registers and written once:
// the kernel moves the bytes it cannot do without and is bound by HBM for
// long inputs, by latency for single tokens. The key rows, which take longer,
// are the first warps of the grid.
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_fp8.h>
#include <cuda_runtime.h>

#include "qsfm_device.cuh"
#include "qsfm_internal.h"

namespace qsfm {
namespace {

constexpr int kRowWarps = 8;
constexpr int kRowThreads = 32 * kRowWarps;
constexpr int kFewRows = 152 * 16;  // query rows up to which a warp has one
constexpr uint32_t kAll = 0xffffffffu;

__device__ __forceinline__ uint32_t bf16x2(float a, float b) {
  const __nv_bfloat162 v = __floats2bfloat162_rn(a, b);
  return *reinterpret_cast<const uint32_t*>(&v);
}
__device__ __forceinline__ float2 of_bf16x2(uint32_t v) {
  return make_float2(__uint_as_float(v << 16), __uint_as_float(v & 0xFFFF0000u));
}
__device__ __forceinline__ float round_bf16(float a) { return __uint_as_float(bf16x2(0.f, a) & 0xFFFF0000u); }

// 8 consecutive elements of an input row as they are read, and in fp32.
template <typename T>
struct Raw {
  uint4 v[sizeof(T) / 2];
  __device__ __forceinline__ void load(const T* src) {
#pragma unroll
    for (int i = 0; i < int(sizeof(T) / 2); ++i) v[i] = reinterpret_cast<const uint4*>(src)[i];
  }
  __device__ __forceinline__ void get(float (&f)[8]) const {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      if constexpr (sizeof(T) == 4) {
        const uint32_t x[8] = {v[0].x, v[0].y, v[0].z, v[0].w, v[1].x, v[1].y, v[1].z, v[1].w};
        f[2 * i] = __uint_as_float(x[2 * i]);
        f[2 * i + 1] = __uint_as_float(x[2 * i + 1]);
      } else {
        const uint32_t x[4] = {v[0].x, v[0].y, v[0].z, v[0].w};
        float2 p;
        if constexpr (__is_same(T, __half)) p = __half22float2(*reinterpret_cast<const __half2*>(&x[i]));
        else p = of_bf16x2(x[i]);
        f[2 * i] = p.x;
        f[2 * i + 1] = p.y;
      }
    }
  }
};
template <typename T>
__device__ __forceinline__ void load8(const T* src, float (&f)[8]) {
  Raw<T> raw;
  raw.load(src);
  raw.get(f);
}

__device__ __forceinline__ void store8_bf16(__nv_bfloat16* dst, const float (&v)[8]) {
  *reinterpret_cast<uint4*>(dst) =
      make_uint4(bf16x2(v[0], v[1]), bf16x2(v[2], v[3]), bf16x2(v[4], v[5]), bf16x2(v[6], v[7]));
}

// The lane's weights (ones without a weight tensor).
__device__ __forceinline__ void load_weights(const void* w, bool bf16, int lane, float (&v)[2][8]) {
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    const int e = 256 * h + 8 * lane;
    if (w == nullptr) {
#pragma unroll
      for (int i = 0; i < 8; ++i) v[h][i] = 1.f;
    } else if (bf16) {
      load8(static_cast<const __nv_bfloat16*>(w) + e, v[h]);
    } else {
      load8(static_cast<const float*>(w) + e, v[h]);
    }
  }
}

// Norm and rotation of the row held by the warp.
__device__ __forceinline__ void norm_rope_row(const qsfm_norm_rope_params& p, bool norm, const float (&w)[2][8],
                                              int pos, int lane, float (&y)[2][8]) {
  if (norm) {
    float sum = 0.f;
#pragma unroll
    for (int h = 0; h < 2; ++h)
#pragma unroll
      for (int i = 0; i < 8; ++i) sum = fmaf(y[h][i], y[h][i], sum);
#pragma unroll
    for (int o = 16; o >= 1; o >>= 1) sum += __shfl_xor_sync(kAll, sum, o);
    const float inv = rsqrtf(sum * (1.f / kDim) + p.eps);
#pragma unroll
    for (int h = 0; h < 2; ++h)
#pragma unroll
      for (int i = 0; i < 8; ++i) y[h][i] *= inv * w[h][i];
  }
  if (p.rope_dim == 0) return;
  const float* table = p.cos_sin + size_t(pos) * p.rope_dim;
  const int half = p.rope_dim / 2;
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    const int r = 256 * h + 8 * lane - p.rope_offset;  // the lane's first element in the rotated range
    const bool in = r >= 0 && r < p.rope_dim;
    if (p.interleaved) {
      if (in) {
        const float4 c = *reinterpret_cast<const float4*>(table + r / 2);
        const float4 s = *reinterpret_cast<const float4*>(table + half + r / 2);
        const float cs[4] = {c.x, c.y, c.z, c.w}, sn[4] = {s.x, s.y, s.z, s.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const float a = y[h][2 * i], b = y[h][2 * i + 1];
          y[h][2 * i] = a * cs[i] - b * sn[i];
          y[h][2 * i + 1] = b * cs[i] + a * sn[i];
        }
      }
    } else if (__any_sync(kAll, in)) {
      // the range starts at a multiple of its (power of two) length, so the
      // other half's lane is this lane with one bit flipped, in the same h
      const bool upper = r >= half;
      const int k = in ? (upper ? r - half : r) : 0;
      float cs[8], sn[8];
      load8(table + k, cs);
      load8(table + half + k, sn);
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const float other = __shfl_xor_sync(kAll, y[h][i], p.rope_dim / 16);
        if (in) y[h][i] = upper ? y[h][i] * cs[i] + other * sn[i] : y[h][i] * cs[i] - other * sn[i];
      }
    }
  }
}

__device__ __forceinline__ float max8(const float (&v)[8]) {
  float m = 0.f;
#pragma unroll
  for (int i = 0; i < 8; ++i) m = fmaxf(m, fabsf(v[i]));
  return m;
}
__device__ __forceinline__ bool finite8(const float (&v)[8]) {
  bool ok = true;
#pragma unroll
  for (int i = 0; i < 8; ++i) ok &= fabsf(v[i]) <= 3.402823466e38f;
  return ok;
}
// floor(log2 x) of a positive normal fp32 (-127 for zero and subnormals)
__device__ __forceinline__ int exponent_of(float x) { return int((__float_as_uint(x) >> 23) & 0xFFu) - 127; }
__device__ __forceinline__ float power_of_two(int e) { return __int_as_float((127 + e) << 23); }  // -126 <= e <= 127

__device__ __forceinline__ uint32_t e4m3x4(float a, float b, float c, float d) {
  const uint32_t lo = __nv_cvt_float2_to_fp8x2(make_float2(a, b), __NV_SATFINITE, __NV_E4M3);
  const uint32_t hi = __nv_cvt_float2_to_fp8x2(make_float2(c, d), __NV_SATFINITE, __NV_E4M3);
  return lo | (hi << 16);
}
__device__ __forceinline__ float of_e4m3(uint32_t code) {
  const __half_raw h = __nv_cvt_fp8_to_halfraw(uint8_t(code), __NV_E4M3);
  return __half2float(*reinterpret_cast<const __half*>(&h));
}
// 8 quotients to e2m1 codes, element 0 in the lowest nibble (nearest even, saturating)
__device__ __forceinline__ uint32_t e2m1x8(const float (&v)[8]) {
  uint32_t r;
  asm("{\n .reg .b8 a, b, c, d;\n"
      " cvt.rn.satfinite.e2m1x2.f32 a, %2, %1;\n cvt.rn.satfinite.e2m1x2.f32 b, %4, %3;\n"
      " cvt.rn.satfinite.e2m1x2.f32 c, %6, %5;\n cvt.rn.satfinite.e2m1x2.f32 d, %8, %7;\n"
      " mov.b32 %0, {a, b, c, d};\n}"
      : "=r"(r)
      : "f"(v[0]), "f"(v[1]), "f"(v[2]), "f"(v[3]), "f"(v[4]), "f"(v[5]), "f"(v[6]), "f"(v[7]));
  return r;
}
__device__ __forceinline__ uint2 dequant8(uint32_t codes, float scale, float (&v)[8]) {
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const uint2 d = dequant4_e2m1(codes >> (16 * i), scale);
    const float2 a = of_bf16x2(d.x), b = of_bf16x2(d.y);
    v[4 * i] = a.x; v[4 * i + 1] = a.y; v[4 * i + 2] = b.x; v[4 * i + 3] = b.y;
  }
  return make_uint2(0, 0);
}

// The warp's row into row `slot` of the cache (slot < 0: nowhere); y becomes
// the values that the stored row stands for.
__device__ __forceinline__ void store_row(const qsfm_norm_rope_params& p, int slot, int lane, float (&y)[2][8]) {
  const bool put = slot >= 0;
  uint8_t* row = static_cast<uint8_t*>(p.kv_cache) + size_t(put ? slot : 0) * kv_row_bytes(p.kv_layout);
  if (p.kv_layout == QSFM_KV_FP8_FP32_SCALES) {
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      float m = max8(y[h]);
#pragma unroll
      for (int o = 1; o <= 4; o <<= 1) m = fmaxf(m, __shfl_xor_sync(kAll, m, o));
      const float scale = __fdiv_rn(fmaxf(m, 1e-12f), 448.f);
      float q[8];
#pragma unroll
      for (int i = 0; i < 8; ++i) q[i] = __fdiv_rn(y[h][i], scale);
      const uint2 code = make_uint2(e4m3x4(q[0], q[1], q[2], q[3]), e4m3x4(q[4], q[5], q[6], q[7]));
      if (put) {
        *reinterpret_cast<uint2*>(row + 256 * h + 8 * lane) = code;
        if ((lane & 7) == 0) p.kv_scale[size_t(slot) * kScales + 4 * h + (lane >> 3)] = scale;
      }
#pragma unroll
      for (int i = 0; i < 8; ++i) y[h][i] = of_e4m3((i < 4 ? code.x : code.y) >> (8 * (i & 3))) * scale;
    }
    return;
  }
  if (p.kv_layout == QSFM_KV_BF16) {
    if (put) {
#pragma unroll
      for (int h = 0; h < 2; ++h) store8_bf16(reinterpret_cast<__nv_bfloat16*>(row) + 256 * h + 8 * lane, y[h]);
    }
    return;
  }
  // packed rows: elements 0..63 (lanes 0..7 of the first half) stay bf16
  const bool rope0 = lane < 8;
  if (p.kv_layout == QSFM_KV_PACKED640) {
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const bool rope = h == 0 && rope0;
      bool ok = finite8(y[h]);
      float m = max8(y[h]);
#pragma unroll
      for (int o = 1; o <= 4; o <<= 1) {
        m = fmaxf(m, __shfl_xor_sync(kAll, m, o));
        ok &= __shfl_xor_sync(kAll, int(ok), o) != 0;
      }
      // the smallest e with m <= 448 2^e = 1.75 2^(e + 8)
      int e = exponent_of(m) - 8;
      if ((__float_as_uint(m) & 0x7FFFFFu) > 0x600000u) ++e;
      e = max(-100, min(100, e));
      const float inv = power_of_two(-e);
      float q[8];
#pragma unroll
      for (int i = 0; i < 8; ++i) q[i] = y[h][i] * inv;
      const uint2 code = make_uint2(e4m3x4(q[0], q[1], q[2], q[3]), e4m3x4(q[4], q[5], q[6], q[7]));
      const int el = 256 * h + 8 * lane;
      if (rope) {
        if (put) store8_bf16(reinterpret_cast<__nv_bfloat16*>(row) + el, y[h]);
#pragma unroll
        for (int i = 0; i < 8; ++i) y[h][i] = round_bf16(y[h][i]);
      } else {
        if (put) {
          *reinterpret_cast<uint2*>(row + 64 + el) = code;
          if ((lane & 7) == 0) row[576 + el / 64 - 1] = ok ? uint8_t(127 + e) : uint8_t(0xFF);
        }
        const float scale = ok ? power_of_two(e) : __uint_as_float(0x7FC00000u);
#pragma unroll
        for (int i = 0; i < 8; ++i) y[h][i] = of_e4m3((i < 4 ? code.x : code.y) >> (8 * (i & 3))) * scale;
      }
    }
    if (put) {  // the padding behind the seven scale bytes
      if (lane == 0) row[583] = 0;
      if (lane < 14) *reinterpret_cast<uint32_t*>(row + 584 + 4 * lane) = 0;
    }
    return;
  }
  // packed384: the row's exponent first, over all 512 elements (finite ones)
  float top = 0.f;
#pragma unroll
  for (int h = 0; h < 2; ++h)
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const float a = fabsf(y[h][i]);
      if (a <= 3.402823466e38f) top = fmaxf(top, a);
    }
#pragma unroll
  for (int o = 16; o >= 1; o >>= 1) top = fmaxf(top, __shfl_xor_sync(kAll, top, o));
  const int e = max(-100, min(100, exponent_of(top) - 10));
  const float power = power_of_two(e), inv_power = power_of_two(-e);
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    const bool rope = h == 0 && rope0;
    const int el = 256 * h + 8 * lane;
    bool ok = finite8(y[h]);
    float m = max8(y[h]);
    m = fmaxf(m, __shfl_xor_sync(kAll, m, 1));
    ok &= __shfl_xor_sync(kAll, int(ok), 1) != 0;
    const float want = __fdiv_rn(m, 6.f) * inv_power;
    const uint32_t s8 = ok ? e4m3x4(want, 0.f, 0.f, 0.f) & 0xFFu : 0x7Fu;
    const float scale = of_e4m3(s8) * power;
    // a division, not a product with the reciprocal: a quotient on a rounding
    // border stays on it
    float q[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) q[i] = scale > 0.f ? __fdiv_rn(y[h][i], scale) : 0.f;
    const uint32_t code = e2m1x8(q);
    if (rope) {
      if (put) store8_bf16(reinterpret_cast<__nv_bfloat16*>(row) + el, y[h]);
#pragma unroll
      for (int i = 0; i < 8; ++i) y[h][i] = round_bf16(y[h][i]);
    } else {
      if (put) {
        *reinterpret_cast<uint32_t*>(row + 128 + (el - 64) / 2) = code;
        if ((lane & 1) == 0) row[352 + (el - 64) / 16] = uint8_t(s8);
      }
      dequant8(code, scale, y[h]);
    }
  }
  if (put && lane == 0) *reinterpret_cast<uint32_t*>(row + 380) = uint32_t(127 + e);
}

// The token's position; false: nothing of the token is read or written.
__device__ __forceinline__ bool token_position(const qsfm_norm_rope_params& p, int t, int* fault, int& pos) {
  pos = p.positions != nullptr ? __ldg(p.positions + t) : 0;
  if (pos < 0) return false;
  if (p.rope_dim != 0 && pos >= p.max_positions) {
    atomicOr(fault, QSFM_FAULT_POSITION);
    return false;
  }
  return true;
}

// kG query rows per warp and turn: their loads are in flight together.
template <typename T, int kG>
__global__ void __launch_bounds__(kRowThreads) norm_rope_kernel(const qsfm_norm_rope_params p, const int kv_blocks,
                                                                int* fault) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  float w[2][8];
  if (int(blockIdx.x) < kv_blocks) {
    load_weights(p.kv_weight, p.weights_bf16 != 0, lane, w);
    for (int t = blockIdx.x * kRowWarps + warp; t < p.tokens; t += kv_blocks * kRowWarps) {
      int pos;
      if (!token_position(p, t, fault, pos)) continue;
      float y[2][8];
      const T* src = static_cast<const T*>(p.kv) + size_t(t) * p.kv_token_stride + 8 * lane;
      load8(src, y[0]);
      load8(src + 256, y[1]);
      int slot = p.kv_cache != nullptr ? __ldg(p.slot_map + t) : -1;
      norm_rope_row(p, p.norm_kv != 0, w, pos, lane, y);
      if (slot >= 0 && (slot >> 7) >= p.num_blocks) {
        atomicOr(fault, QSFM_FAULT_SLOT);
        slot = -1;
      }
      store_row(p, slot, lane, y);
      if (p.kv_out != nullptr) {
        __nv_bfloat16* out = static_cast<__nv_bfloat16*>(p.kv_out) + size_t(t) * kDim + 8 * lane;
        store8_bf16(out, y[0]);
        store8_bf16(out + 256, y[1]);
      }
    }
    return;
  }
  load_weights(p.q_weight, p.weights_bf16 != 0, lane, w);
  const int rows = p.tokens * p.heads, step = (gridDim.x - kv_blocks) * kRowWarps * kG;
  for (int r0 = ((blockIdx.x - kv_blocks) * kRowWarps + warp) * kG; r0 < rows; r0 += step) {
    Raw<T> raw[kG][2];
    int pos[kG];
    bool live[kG];
    const int t0 = r0 / p.heads, head0 = r0 - t0 * p.heads;
#pragma unroll
    for (int g = 0; g < kG; ++g) {
      int t = t0, head = head0 + g;
      while (head >= p.heads) {  // at most kG turns
        head -= p.heads;
        ++t;
      }
      live[g] = r0 + g < rows;
      if (!live[g]) continue;
      pos[g] = p.positions != nullptr ? __ldg(p.positions + t) : 0;
      const T* src = static_cast<const T*>(p.q) + size_t(t) * p.q_token_stride + size_t(head) * p.q_head_stride + 8 * lane;
      raw[g][0].load(src);
      raw[g][1].load(src + 256);
    }
#pragma unroll
    for (int g = 0; g < kG; ++g) {
      if (!live[g] || pos[g] < 0) continue;
      if (p.rope_dim != 0 && pos[g] >= p.max_positions) {
        if (lane == 0) atomicOr(fault, QSFM_FAULT_POSITION);
        continue;
      }
      float y[2][8];
      raw[g][0].get(y[0]);
      raw[g][1].get(y[1]);
      norm_rope_row(p, p.norm_q != 0, w, pos[g], lane, y);
      __nv_bfloat16* out = static_cast<__nv_bfloat16*>(p.q_out) + size_t(r0 + g) * kDim + 8 * lane;
      store8_bf16(out, y[0]);
      store8_bf16(out + 256, y[1]);
    }
  }
}

template <typename T>
void launch_rows(const qsfm_norm_rope_params& p, int* fault, cudaStream_t s) {
  auto blocks = [](long long warps) { return int((warps + kRowWarps - 1) / kRowWarps); };
  const int kv_blocks = p.kv != nullptr ? min(blocks(p.tokens), 1 << 14) : 0;
  const long long rows = p.q != nullptr ? (long long)p.tokens * p.heads : 0;
  // Few rows: one per warp, as many warps as rows (latency). Many: four per
  // turn (two of fp32), so that a warp's loads overlap.
  constexpr int kG = sizeof(T) == 4 ? 2 : 4;
  if (rows <= kFewRows)
    norm_rope_kernel<T, 1><<<kv_blocks + blocks(rows), kRowThreads, 0, s>>>(p, kv_blocks, fault);
  else
    norm_rope_kernel<T, kG><<<kv_blocks + min(blocks((rows + kG - 1) / kG), 1 << 14), kRowThreads, 0, s>>>(p, kv_blocks, fault);
}

}  // namespace

cudaError_t launch_norm_rope(const qsfm_norm_rope_params& p, int* fault, cudaStream_t s) {
  if (p.in_type == QSFM_F32) launch_rows<float>(p, fault, s);
  else if (p.in_type == QSFM_F16) launch_rows<__half>(p, fault, s);
  else launch_rows<__nv_bfloat16>(p, fault, s);
  return cudaGetLastError();
}

}  // namespace qsfm
