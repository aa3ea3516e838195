// Norm, position rotation and cache store of query and key rows (sm_103a).
//
// For each head row x of a token (512 elements):
//   y = x / sqrt(mean(x^2) + eps) * weight, then the rope_dim elements from
//   rope_offset on are turned by the token's angles,
// rounded once: queries to bf16, the token's one latent key row to its cache
// row format (bf16, e4m3 with fp32 or e8m0 scales, e2m1 with e4m3 scales).
//
// One warp per row: lane l holds elements 8 l .. + 7 of each 256-element half
// (two 16-byte vectors of a bf16 row), so the sum of squares is five shuffles,
// the pairs of a rotation are in the lane (adjacent) or rope_dim / 16 lanes
// apart (halves), and a quantisation group of 16 or 64 elements is 2 or 8
// neighbouring lanes. A row is read once, held in registers and written once.
// Query rows are bound by HBM, so what counts is bytes in flight: a warp streams
// its rows through a ring in shared memory. The key rows are few; they are the
// first blocks of the grid, one warp each, bound by latency and by the
// instructions of their last bits (below).
// Measured inside a graph: 4099 tokens of 128 + 1 bf16 rows 177 us, 6.1 TB/s of rows
// read and written (90% of a copy's rate); 256 tokens 6.5 us; one token 3.9 us; 8191
// fp32 key rows alone, fp8 rows stored, 12.9 us.
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
constexpr int kRowBlocks = 3;  // blocks on an SM
// query rows a warp has in flight: 8 KB (1 KB a row, fp32 2 KB)
template <typename T>
constexpr int stages() {
  return sizeof(T) == 4 ? 4 : 8;
}
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

// (streaming: the rows are not read again here; 256 tokens 7.4 -> 6.3 us)
__device__ __forceinline__ void store8_bf16(__nv_bfloat16* dst, const float (&v)[8]) {
  __stcs(reinterpret_cast<uint4*>(dst),
      make_uint4(bf16x2(v[0], v[1]), bf16x2(v[2], v[3]), bf16x2(v[4], v[5]), bf16x2(v[6], v[7])));
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

// The lane's cosines and sines for a token: interleaved pairs use four of each,
// halves eight. `h`: the half row that holds the rotated range (a range never
// crosses the middle: it starts at a multiple of its power-of-two length).
struct Turn {
  float c[8], s[8];
};
__device__ __forceinline__ int rotated_half(const qsfm_norm_rope_params& p) { return p.rope_offset >> 8; }
__device__ __forceinline__ int rotated_element(const qsfm_norm_rope_params& p, int lane) {
  return 8 * lane + (p.rope_offset & ~255) - p.rope_offset;  // the lane's first, counted from the range's start
}
__device__ __forceinline__ void load_turn(const qsfm_norm_rope_params& p, int pos, int lane, Turn& t) {
  const int r = rotated_element(p, lane), half = p.rope_dim / 2;
  if (r < 0 || r >= p.rope_dim) return;
  const float* table = p.cos_sin + size_t(pos) * p.rope_dim;
  if (p.interleaved) {
    const float4 c = *reinterpret_cast<const float4*>(table + r / 2);
    const float4 s = *reinterpret_cast<const float4*>(table + half + r / 2);
    t.c[0] = c.x; t.c[1] = c.y; t.c[2] = c.z; t.c[3] = c.w;
    t.s[0] = s.x; t.s[1] = s.y; t.s[2] = s.z; t.s[3] = s.w;
  } else {
    const int k = r >= half ? r - half : r;
    load8(table + k, t.c);
    load8(table + half + k, t.s);
  }
}
__device__ __forceinline__ void turn8(const qsfm_norm_rope_params& p, int lane, const Turn& t, float (&y)[8]) {
  const int r = rotated_element(p, lane);
  const bool in = r >= 0 && r < p.rope_dim;
  if (p.interleaved) {
    if (in) {
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const float a = y[2 * i], b = y[2 * i + 1];
        y[2 * i] = a * t.c[i] - b * t.s[i];
        y[2 * i + 1] = b * t.c[i] + a * t.s[i];
      }
    }
  } else {
    // the other half's lane is this lane with one bit flipped
    const bool upper = r >= p.rope_dim / 2;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const float other = __shfl_xor_sync(kAll, y[i], p.rope_dim / 16);
      if (in) y[i] = upper ? y[i] * t.c[i] + other * t.s[i] : y[i] * t.c[i] - other * t.s[i];
    }
  }
}

__device__ __forceinline__ float inverse_rms(const qsfm_norm_rope_params& p, const float (&y)[2][8]) {
  float sum = 0.f;
#pragma unroll
  for (int h = 0; h < 2; ++h)
#pragma unroll
    for (int i = 0; i < 8; ++i) sum = fmaf(y[h][i], y[h][i], sum);
#pragma unroll
  for (int o = 16; o >= 1; o >>= 1) sum += __shfl_xor_sync(kAll, sum, o);
  return rsqrtf(sum * (1.f / kDim) + p.eps);
}
// Norm and rotation of the row held by the warp.
__device__ __forceinline__ void norm_rope_row(const qsfm_norm_rope_params& p, bool norm, const float (&w)[2][8],
                                              const Turn& turn, int lane, float (&y)[2][8]) {
  if (norm) {
    const float inv = inverse_rms(p, y);
#pragma unroll
    for (int h = 0; h < 2; ++h)
#pragma unroll
      for (int i = 0; i < 8; ++i) y[h][i] *= inv * w[h][i];
  }
  if (p.rope_dim == 0) return;
  if (rotated_half(p) == 0) turn8(p, lane, turn, y[0]);
  else turn8(p, lane, turn, y[1]);
}

// ------------------------------------------------------------- key rows
// A stored row is rounded to few bits, so what matters is on which side of a
// rounding border a value lies: key rows are computed as y + z, z what fp32 y
// leaves over. In 8191 rows of 512 that are stored as bf16 fp32 alone puts 50
// elements on the wrong side, and 3 to 6 of the codes of the other formats; this
// none. It costs the key rows half of their time (8191 fp32 rows 7.9 -> 12.0 us,
// one token 3.1 -> 3.6 us); the query rows, whose results are not stored codes, go
// without. The sum and the product with what they leave over are Knuth's and Dekker's
// error-free transformations (the product's rest by a fused multiply-add).
__device__ __forceinline__ void two_sum(float a, float b, float& s, float& e) {
  s = a + b;
  const float t = s - a;
  e = (a - (s - t)) + (b - t);
}
__device__ __forceinline__ void two_product(float a, float b, float& p, float& e) {
  p = __fmul_rn(a, b);
  e = fmaf(a, b, -p);
}
// h + t as y + z; of an h that is not finite nothing is left
__device__ __forceinline__ void renormed(float h, float t, float& y, float& z) {
  if (!(fabsf(t) <= 3.402823466e38f)) t = 0.f;
  y = h + t;
  z = t - (y - h);
}
// a c + b d for a + az, b + bz
__device__ __forceinline__ void turned(float a, float az, float c, float b, float bz, float d, float& y, float& z) {
  float u, ue, v, ve, h, t;
  two_product(a, c, u, ue);
  two_product(b, d, v, ve);
  two_sum(u, v, h, t);
  t += fmaf(az, c, ue) + fmaf(bz, d, ve);
  renormed(h, t, y, z);
}
__device__ __forceinline__ void turn8(const qsfm_norm_rope_params& p, int lane, const Turn& t, float (&y)[8],
                                      float (&z)[8]) {
  const int r = rotated_element(p, lane);
  const bool in = r >= 0 && r < p.rope_dim;
  if (p.interleaved) {
    if (in) {
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const float a = y[2 * i], az = z[2 * i], b = y[2 * i + 1], bz = z[2 * i + 1];
        turned(a, az, t.c[i], b, bz, -t.s[i], y[2 * i], z[2 * i]);
        turned(b, bz, t.c[i], a, az, t.s[i], y[2 * i + 1], z[2 * i + 1]);
      }
    }
  } else {
    const bool upper = r >= p.rope_dim / 2;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const float other = __shfl_xor_sync(kAll, y[i], p.rope_dim / 16), oz = __shfl_xor_sync(kAll, z[i], p.rope_dim / 16);
      if (in) turned(y[i], z[i], t.c[i], other, oz, upper ? t.s[i] : -t.s[i], y[i], z[i]);
    }
  }
}
template <bool kExactSquares>  // of 16-bit inputs
__device__ __forceinline__ void norm_rope_row(const qsfm_norm_rope_params& p, bool norm, const float (&w)[2][8],
                                              const Turn& turn, int lane, float (&y)[2][8], float (&z)[2][8]) {
#pragma unroll
  for (int h = 0; h < 2; ++h)
#pragma unroll
    for (int i = 0; i < 8; ++i) z[h][i] = 0.f;
  if (norm) {
    float inv, inv_rest = 0.f;
    if (p.kv_layout == QSFM_KV_FP8_FP32_SCALES) {
      inv = inverse_rms(p, y);  // common to a value and its group's scale: no code depends on its last bits
    } else {
      float sum = 0.f, rest = 0.f;
#pragma unroll
      for (int h = 0; h < 2; ++h)
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          float q, e, t;
          two_product(y[h][i], y[h][i], q, e);
          two_sum(sum, q, sum, t);
          rest += kExactSquares ? t : t + e;
        }
#pragma unroll
      for (int o = 16; o >= 1; o >>= 1) {
        float t;
        const float other = __shfl_xor_sync(kAll, sum, o), other_rest = __shfl_xor_sync(kAll, rest, o);
        two_sum(sum, other, sum, t);
        rest = (rest + other_rest) + t;
      }
      float mean, t, q, e;
      two_sum(sum * (1.f / kDim), p.eps, mean, t);
      rest = fmaf(rest, 1.f / kDim, t);
      // one step of Newton's method from the fp32 root: inv + inv_rest
      inv = rsqrtf(mean);
      two_product(inv, inv, q, e);
      const float off = fmaf(-mean, q, 1.f) - fmaf(mean, e, rest * q);
      inv_rest = 0.5f * inv * off;
    }
#pragma unroll
    for (int h = 0; h < 2; ++h)
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        float a, b, u, v;
        two_product(inv, w[h][i], a, b);
        b = fmaf(inv_rest, w[h][i], b);
        two_product(y[h][i], a, u, v);
        v = fmaf(y[h][i], b, v);
        renormed(u, v, y[h][i], z[h][i]);
      }
  }
  if (p.rope_dim == 0) return;
  if (rotated_half(p) == 0) turn8(p, lane, turn, y[0], z[0]);
  else turn8(p, lane, turn, y[1], z[1]);
}

// y + z in fp32 for a rounding to at most 22 bits: what is left over sets the
// last bit, so the value lies on a border only where y + z does.
__device__ __forceinline__ float sticky(float y, float z) {
  const uint32_t b = __float_as_uint(y);
  const bool rest = fabsf(z) > 0.f && fabsf(y) <= 3.402823466e38f;
  return rest ? __uint_as_float(((y < 0.f) == (z < 0.f) ? b : b - 1) | 1u) : y;
}
__device__ __forceinline__ void sticky16(float (&y)[2][8], const float (&z)[2][8]) {
#pragma unroll
  for (int h = 0; h < 2; ++h)
#pragma unroll
    for (int i = 0; i < 8; ++i) y[h][i] = sticky(y[h][i], z[h][i]);
}
// (y + z) / (d + dz), d > 0, all finite, in the same sense, for a rounding to at most 18 bits: the
// quotient by the reciprocal (two ulps off at most) goes to the next multiple of
// 16 ulps, and the sign of what is left over says on which side of it y + z is.
__device__ __forceinline__ float sticky_quotient(float y, float z, float d, float dz, float reciprocal) {
  const float a = fabsf(y);
  uint32_t b = (__float_as_uint(a * reciprocal) + 8u) & ~15u;
  const float q = __uint_as_float(b), left = fmaf(-q, d, a) + fmaf(-q, dz, y < 0.f ? -z : z);
  if (left < 0.f && b > 0) b -= 1;
  if (left < 0.f || left > 0.f) b |= 1u;
  return copysignf(__uint_as_float(b), y);
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
__device__ __forceinline__ void dequant8(uint32_t codes, float scale, float (&v)[8]) {
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const uint2 d = dequant4_e2m1(codes >> (16 * i), scale);
    const float2 a = of_bf16x2(d.x), b = of_bf16x2(d.y);
    v[4 * i] = a.x; v[4 * i + 1] = a.y; v[4 * i + 2] = b.x; v[4 * i + 3] = b.y;
  }
}

// The warp's row y + z into row `slot` of the cache (slot < 0: nowhere); y becomes
// the values that the stored row stands for.
__device__ __forceinline__ void store_row(const qsfm_norm_rope_params& p, int slot, int lane, float (&y)[2][8],
                                          const float (&z)[2][8]) {
  const bool put = slot >= 0;
  uint8_t* row = static_cast<uint8_t*>(p.kv_cache) + size_t(put ? slot : 0) * kv_row_bytes(p.kv_layout);
  if (p.kv_layout == QSFM_KV_FP8_FP32_SCALES) {
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      bool ok = finite8(y[h]);
#pragma unroll
      for (int o = 1; o <= 4; o <<= 1) ok &= __shfl_xor_sync(kAll, int(ok), o) != 0;
      float m = 0.f, rest = 0.f;  // the largest |y + z|
      auto larger = [&](float a, float az) {
        if (a > m || (a == m && az > rest)) m = a, rest = az;
      };
#pragma unroll
      for (int i = 0; i < 8; ++i) larger(fabsf(y[h][i]), y[h][i] < 0.f ? -z[h][i] : z[h][i]);
#pragma unroll
      for (int o = 1; o <= 4; o <<= 1) {
        const float a = __shfl_xor_sync(kAll, m, o), az = __shfl_xor_sync(kAll, rest, o);
        larger(a, az);
      }
      if (m <= 1e-12f) m = 1e-12f, rest = 0.f;
      float scale = m * (1.f / 448.f);
      const float off = fmaf(-scale, 448.f, m) + rest;
      float scale_rest = 0.f;  // codes go by max|y| / 448 itself, of which `scale` is the rounding
      if (fabsf(off) <= 3.402823466e38f) {
        scale = fmaf(off, 1.f / 448.f, scale);
        scale_rest = (fmaf(-scale, 448.f, m) + rest) * (1.f / 448.f);
      }
      const float reciprocal = __frcp_rn(scale);
      float q[8];
#pragma unroll
      for (int i = 0; i < 8; ++i) q[i] = sticky_quotient(y[h][i], z[h][i], scale, scale_rest, reciprocal);
      uint2 code = make_uint2(e4m3x4(q[0], q[1], q[2], q[3]), e4m3x4(q[4], q[5], q[6], q[7]));
      if (!ok) {  // NaN codes as well as a NaN scale: a reader may limit the scale
        code = make_uint2(0x7F7F7F7Fu, 0x7F7F7F7Fu);
        scale = __uint_as_float(0x7FC00000u);
      }
      if (put) {
        *reinterpret_cast<uint2*>(row + 256 * h + 8 * lane) = code;
        if ((lane & 7) == 0) p.kv_scale[size_t(slot) * kScales + 4 * h + (lane >> 3)] = scale;
      }
#pragma unroll
      for (int i = 0; i < 8; ++i) y[h][i] = of_e4m3((i < 4 ? code.x : code.y) >> (8 * (i & 3))) * scale;
    }
    return;
  }
  sticky16(y, z);
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
    const float want = sticky_quotient(m, 0.f, 6.f, 0.f, 1.f / 6.f) * inv_power;
    const uint32_t s8 = ok ? e4m3x4(want, 0.f, 0.f, 0.f) & 0xFFu : 0x7Fu;
    const float scale = of_e4m3(s8) * power;
    const float reciprocal = scale > 0.f ? __frcp_rn(scale) : 0.f;
    float q[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) q[i] = scale > 0.f ? sticky_quotient(y[h][i], 0.f, scale, 0.f, reciprocal) : 0.f;
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

__device__ __forceinline__ int position_of(const qsfm_norm_rope_params& p, int t) {
  return p.positions != nullptr ? __ldg(p.positions + t) : 0;
}
// False: nothing is written for the token (padding, or a position past the table).
__device__ __forceinline__ bool position_ok(const qsfm_norm_rope_params& p, int pos, int lane, int* fault) {
  if (pos < 0) return false;
  if (p.rope_dim != 0 && pos >= p.max_positions) {
    if (lane == 0) atomicOr(fault, QSFM_FAULT_POSITION);
    return false;
  }
  return true;
}

__device__ __forceinline__ void copy_async16(uint32_t dst, const void* src) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
}

// Blocks 0 .. kv_blocks - 1: one key row per warp, its input, position and slot
// requested together. The others: query rows, `per` consecutive ones per block.
// A warp streams them through a ring of its own in shared memory, kStages rows
// in flight (asynchronous copies; each lane reads back only what it copied, so
// no barrier), and keeps the token's cosines and sines from head to head.
template <typename T>
__global__ void __launch_bounds__(kRowThreads, kRowBlocks)
    norm_rope_kernel(const qsfm_norm_rope_params p, const int kv_blocks, const int per, int* fault) {
  extern __shared__ __align__(16) uint8_t s_rows[];
  constexpr int kStages = stages<T>();
  constexpr int kVec = sizeof(T) / 2;  // 16-byte vectors of 8 elements
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  float w[2][8], y[2][8];
  Turn turn;
  if (int(blockIdx.x) < kv_blocks) {
    const int t = blockIdx.x * kRowWarps + warp;
    if (t >= p.tokens) return;
    const T* src = static_cast<const T*>(p.kv) + size_t(t) * p.kv_token_stride + 8 * lane;
    const int pos = position_of(p, t);
    int slot = p.kv_cache != nullptr ? __ldg(p.slot_map + t) : -1;
    Raw<T> raw[2];
    raw[0].load(src);
    raw[1].load(src + 256);
    load_weights(p.kv_weight, p.weights_bf16 != 0, lane, w);
    if (!position_ok(p, pos, lane, fault)) return;
    if (p.rope_dim != 0) load_turn(p, pos, lane, turn);
    raw[0].get(y[0]);
    raw[1].get(y[1]);
    float z[2][8];
    norm_rope_row<sizeof(T) == 2>(p, p.norm_kv != 0, w, turn, lane, y, z);
    if (slot >= 0 && (slot >> 7) >= p.num_blocks) {
      if (lane == 0) atomicOr(fault, QSFM_FAULT_SLOT);
      slot = -1;
    }
    store_row(p, slot, lane, y, z);
    if (p.kv_out != nullptr) {
      __nv_bfloat16* out = static_cast<__nv_bfloat16*>(p.kv_out) + size_t(t) * kDim + 8 * lane;
      store8_bf16(out, y[0]);
      store8_bf16(out + 256, y[1]);
    }
    return;
  }
  const int rows = p.tokens * p.heads;
  // `per` rows of the block, its warps side by side: a turn of the block is
  // contiguous where q is
  const int b0 = (blockIdx.x - kv_blocks) * per, r0 = b0 + warp, r1 = min(rows, b0 + per);
  if (r0 >= r1) return;
  // row r as (token, head), advanced by the block's warps
  int t_in = r0 / p.heads, head_in = r0 - t_in * p.heads;
  int t = t_in, head = head_in;
  const uint32_t ring = smem_u32(s_rows) + uint32_t(warp * kStages) * kDim * sizeof(T) + 16 * lane;
  auto request = [&](int r) {
    if (r < r1) {
      const T* src = static_cast<const T*>(p.q) + size_t(t_in) * p.q_token_stride +
                     size_t(head_in) * p.q_head_stride + 8 * lane;
      const uint32_t dst = ring + uint32_t((r - r0) / kRowWarps % kStages) * kDim * sizeof(T);
#pragma unroll
      for (int h = 0; h < 2; ++h)
#pragma unroll
        for (int i = 0; i < kVec; ++i)
          copy_async16(dst + uint32_t(h * kVec + i) * 512, reinterpret_cast<const uint4*>(src + 256 * h) + i);
      head_in += kRowWarps;
      while (head_in >= p.heads) {
        head_in -= p.heads;
        ++t_in;
      }
    }
    asm volatile("cp.async.commit_group;" ::: "memory");
  };
#pragma unroll
  for (int i = 0; i < kStages - 1; ++i) request(r0 + i * kRowWarps);
  int pos = position_of(p, t);
  load_weights(p.q_weight, p.weights_bf16 != 0, lane, w);
  bool ok = position_ok(p, pos, lane, fault);
  if (ok && p.rope_dim != 0) load_turn(p, pos, lane, turn);
  for (int r = r0; r < r1; r += kRowWarps) {
    request(r + (kStages - 1) * kRowWarps);
    asm volatile("cp.async.wait_group %0;" ::"n"(kStages - 1) : "memory");
    if (ok) {
      const uint32_t src = ring + uint32_t((r - r0) / kRowWarps % kStages) * kDim * sizeof(T);
      Raw<T> raw[2];
#pragma unroll
      for (int h = 0; h < 2; ++h)
#pragma unroll
        for (int i = 0; i < kVec; ++i) raw[h].v[i] = lds_v4(src + uint32_t(h * kVec + i) * 512);
      raw[0].get(y[0]);
      raw[1].get(y[1]);
      norm_rope_row(p, p.norm_q != 0, w, turn, lane, y);
      __nv_bfloat16* out = static_cast<__nv_bfloat16*>(p.q_out) + size_t(r) * kDim + 8 * lane;
      store8_bf16(out, y[0]);
      store8_bf16(out + 256, y[1]);
    }
    head += kRowWarps;
    if (head >= p.heads && r + kRowWarps < r1) {
      while (head >= p.heads) {
        head -= p.heads;
        ++t;
      }
      pos = position_of(p, t);
      ok = position_ok(p, pos, lane, fault);
      if (ok && p.rope_dim != 0) load_turn(p, pos, lane, turn);
    }
  }
}

template <typename T>
cudaError_t launch_rows(const qsfm_norm_rope_params& p, int* fault, cudaStream_t s) {
  const int kv_blocks = p.kv != nullptr ? (p.tokens + kRowWarps - 1) / kRowWarps : 0;
  if (p.q == nullptr) {
    norm_rope_kernel<T><<<kv_blocks, kRowThreads, 0, s>>>(p, kv_blocks, 0, fault);
    return cudaGetLastError();
  }
  constexpr int kSmem = kRowWarps * stages<T>() * kDim * int(sizeof(T));
  cudaError_t e = cudaFuncSetAttribute(norm_rope_kernel<T>, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmem);
  int dev = 0, sms = 0;
  if (e == cudaSuccess) e = cudaGetDevice(&dev);
  if (e == cudaSuccess) e = cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
  if (e != cudaSuccess) return e;
  const int rows = p.tokens * p.heads;
  // as many blocks of query rows as run at once, and their share of the rows
  const int blocks = sms * kRowBlocks;
  int per = (rows + blocks - 1) / blocks;
  per = (per + kRowWarps - 1) / kRowWarps * kRowWarps;
  const int q_blocks = (rows + per - 1) / per;
  norm_rope_kernel<T><<<kv_blocks + q_blocks, kRowThreads, kSmem, s>>>(p, kv_blocks, per, fault);
  return cudaGetLastError();
}

}  // namespace

cudaError_t launch_norm_rope(const qsfm_norm_rope_params& p, int* fault, cudaStream_t s) {
  return p.in_type == QSFM_F32   ? launch_rows<float>(p, fault, s)
         : p.in_type == QSFM_F16 ? launch_rows<__half>(p, fault, s)
                                 : launch_rows<__nv_bfloat16>(p, fault, s);
}

}  // namespace qsfm
