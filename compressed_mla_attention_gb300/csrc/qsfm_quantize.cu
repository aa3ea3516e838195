// Rows quantised to e4m3 with one fp32 scale per 128 elements (sm_103a).
//
// For each group of 128 elements y of a row, with A = max|y|:
//   scale = A / 448, code = e4m3(448 y / A) to nearest even, A at least 1e-12, or, with
//   scales that are powers of two, scale = 2^e of the smallest e with A <= 448 2^e.
// y is the input itself, the input times silu(gate), or the input with a part of
// each head turned by its position's angles; a row may be taken from anywhere in
// the input (row_index).
//
// Eight lanes hold a group, each two runs of eight elements (8 l and 64 + 8 l), so that
// a load of a 16-bit input is whole lines, A is three shuffles, and a pair of a rotation
// is in the lane (adjacent, or 64 elements apart) or rope_dim / 16 lanes away. The kernel
// is bound by HBM as long as it takes few instructions: with sixteen elements a lane what
// is done once a group weighs little.
//
// Every code is the formula's, by one of two ways.
//  * Where y and A are 16-bit inputs as they are, 448 y / A either lies on the border of
//    two codes or is 2^-17 of itself away from it (y and A have at most 11 significant
//    bits, a border five). These borders are met all the time: with bf16 inputs in a
//    quarter of the groups. The quotient is made a little too large, by 2 to 10 units of
//    2^-24, and its last four bits are cut: what lies on a border is then on it, what
//    does not stays on its side.
//  * Elsewhere (y computed, or fp32) an element is next to a border by chance. The
//    quotient, within a few units (`error` in finish()), is converted twice, times 1 - error and
//    1 + error: where both give the same code, that is the code. Otherwise the sign of
//    448 |y| - m A decides, m the border (0: the even code), with y and A as sums of two
//    fp32 values and the products' roundings carried: about 46 bits (of the terms, where a
//    turned y is a small difference of large ones).
//
// Measured (a call among others in a graph): 16384 bf16 rows of 8192 in 62 us, 6.6 TB/s,
// the rate of a copy; 4099 tokens of 64 heads of 512, 64 elements of each turned, 88 us,
// 4.7 TB/s (the launch of the turned groups takes 26 instructions an element, two thirds of
// the issue slots of its 36 us; the other moves 5.4 TB/s); gated 32 us, 5.2 TB/s, 0.6 of
// the issue slots; one row 1.2 us.
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include <type_traits>

#include "qsfm_device.cuh"
#include "qsfm_divide.cuh"
#include "qsfm_internal.h"

namespace qsfm {
namespace {

constexpr int kQGroup = 128;        // elements of a scale
constexpr int kQLanes = 8;          // lanes of a group
constexpr int kQElems = 16;         // elements of a lane
constexpr int kQWarps = 8;
constexpr uint32_t kAllLanes = 0xffffffffu;
constexpr float kQMin = 1e-12f;     // A of an all-zero group,
constexpr float kQMinRest = float(1e-12 - double(kQMin));  // and what fp32 leaves over of it

enum QuantizeMode { kPlain = 0, kAdjacent = 1, kHalves = 2, kGated = 3 };  // the middle two turn pairs

// Blocks on an SM, from what was measured: 16384 bf16 rows of 8192 in 62 us with 6, 65 with
// 4; 16001 gated rows of 2048 in 32 us with 5, 33 with 4; 4099 x 64 turned heads of 512 in 88 us
// with 4, 93 with 5 or 3.
constexpr int blocks_per_sm(int mode) { return mode == kPlain ? 6 : mode == kGated ? 5 : 4; }

struct QuantizeShape {
  uint32_t groups;   // scales of a row
  uint32_t total;    // rows * groups
  int k;             // elements of a row
  uint32_t units;    // fours of groups that a warp takes at a time
  FastDiv groups_of; // by the groups of a row (kHeads: by those of a head row that a launch takes)
  FastDiv heads_of;  // kHeads: by the heads; else by the groups of a head row
  uint32_t of_head;  // kHeads: groups of a head row; those from first on, without the one at skip
  uint32_t first, skip;
};

// 8 consecutive elements as they are read, and in fp32.
template <typename T>
struct Eight {
  uint4 v[sizeof(T) / 2];
  __device__ __forceinline__ void load(const T* src) {
#pragma unroll
    for (int i = 0; i < int(sizeof(T) / 2); ++i) v[i] = ldg_nc_v4(reinterpret_cast<const uint4*>(src) + i);
  }
  __device__ __forceinline__ void zero() {
#pragma unroll
    for (int i = 0; i < int(sizeof(T) / 2); ++i) v[i] = make_uint4(0, 0, 0, 0);
  }
  __device__ __forceinline__ void get(float* f) const {
    if constexpr (sizeof(T) == 4) {
      const uint32_t x[8] = {v[0].x, v[0].y, v[0].z, v[0].w, v[1].x, v[1].y, v[1].z, v[1].w};
#pragma unroll
      for (int i = 0; i < 8; ++i) f[i] = __uint_as_float(x[i]);
    } else {
      const uint32_t x[4] = {v[0].x, v[0].y, v[0].z, v[0].w};
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        if constexpr (std::is_same<T, __half>::value) {
          const float2 p = __half22float2(*reinterpret_cast<const __half2*>(&x[i]));
          f[2 * i] = p.x;
          f[2 * i + 1] = p.y;
        } else {
          f[2 * i] = __uint_as_float(x[i] << 16);
          f[2 * i + 1] = __uint_as_float(x[i] & 0xFFFF0000u);
        }
      }
    }
  }
};

// max(|a|, |b|), NaN when one is.
__device__ __forceinline__ float abs_max(float a, float b) {
  float r;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(fabsf(a)), "f"(fabsf(b)));
  return r;
}

// (a, b) * r, both products in one instruction.
__device__ __forceinline__ float2 mul2(float a, float b, float r) {
  float2 o;
  asm("{\n .reg .b64 x, y, z;\n mov.b64 x, {%2, %3};\n mov.b64 y, {%4, %4};\n mul.rn.f32x2 z, x, y;\n"
      " mov.b64 {%0, %1}, z;\n}"
      : "=f"(o.x), "=f"(o.y)
      : "f"(a), "f"(b), "f"(r));
  return o;
}

// e4m3 codes of a (low byte), b, c, d, to nearest even, saturating.
__device__ __forceinline__ uint32_t e4m3x4(float a, float b, float c, float d) {
  uint32_t r;
  asm("{\n .reg .b16 lo, hi;\n cvt.rn.satfinite.e4m3x2.f32 lo, %2, %1;\n cvt.rn.satfinite.e4m3x2.f32 hi, %4, %3;\n"
      " mov.b32 %0, {lo, hi};\n}"
      : "=r"(r)
      : "f"(a), "f"(b), "f"(c), "f"(d));
  return r;
}
// Codes of y r; kCut: of the products without their last four bits.
template <bool kCut>
__device__ __forceinline__ void codes16(const float (&y)[kQElems], float r, uint32_t (&c)[4]) {
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    float2 a = mul2(y[4 * i], y[4 * i + 1], r), b = mul2(y[4 * i + 2], y[4 * i + 3], r);
    if constexpr (kCut) {
      a.x = __uint_as_float(__float_as_uint(a.x) & ~15u);
      a.y = __uint_as_float(__float_as_uint(a.y) & ~15u);
      b.x = __uint_as_float(__float_as_uint(b.x) & ~15u);
      b.y = __uint_as_float(__float_as_uint(b.y) & ~15u);
    }
    c[i] = e4m3x4(a.x, a.y, b.x, b.y);
  }
}

// 1 / a within 1 unit in the last place (a and the result normal).
__device__ __forceinline__ float rcp_approx(float a) {
  float r;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(a));
  return r;
}
// a / 448 to nearest: a quotient by the reciprocal, corrected by its remainder, is the
// rounded one (Markstein's theorem, the reciprocal being rounded to nearest).
__device__ __forceinline__ float over448(float a) {
  constexpr float kInv = 1.0f / 448.0f;
  const float q = a * kInv;
  return __fmaf_rn(__fmaf_rn(-448.f, q, a), kInv, q);
}

// The smallest e with a + more <= 448 2^e = 1.75 2^(8 + e), within -100 .. 100 (|more| at
// most half a unit of a).
__device__ __forceinline__ int pow2_exponent(float a, float more = 0.f) {
  const uint32_t u = __float_as_uint(a), part = u & 0x7FFFFFu;
  return min(max(int(u >> 23) - 127 - 8 + (part > 0x600000u || (part == 0x600000u && more > 0.f) ? 1 : 0), -100), 100);
}
__device__ __forceinline__ float power2(int e) { return __uint_as_float(uint32_t(e + 127) << 23); }

// A value as the sum of two fp32 numbers, the second at most half a unit of the first.
struct Wide {
  float hi, lo;
};

// a c - b s by Kahan's difference of products: with what its roundings leave over (each
// result within 1.5 units), so that y is as good where its terms cancel.
__device__ __forceinline__ float turned(float a, float c, float b, float s) {
  const float w = b * s;
  return __fmaf_rn(a, c, -w) + __fmaf_rn(-b, s, w);
}
// The same to about 2^-46 of the terms: both products and their difference exact, what
// is left over added in fp32.
__device__ __forceinline__ Wide turned_wide(float a, float c, float b, float s) {
  const float v = a * c, w = b * s;
  const float d = v - w, part = d - v;
  const float left = (v - (d - part)) - (w + part);  // v - w - d
  const float e = left + (__fmaf_rn(a, c, -v) - __fmaf_rn(b, s, -w));
  const float h = d + e;
  return {h, e - (h - d)};
}

// (a, b) + 1.
__device__ __forceinline__ float2 plus1(float2 v) {
  float2 o;
  asm("{\n .reg .b64 x, y, z;\n mov.b64 x, {%2, %3};\n mov.b64 y, {%4, %4};\n add.rn.f32x2 z, x, y;\n"
      " mov.b64 {%0, %1}, z;\n}"
      : "=f"(o.x), "=f"(o.y)
      : "f"(v.x), "f"(v.y), "f"(1.f));
  return o;
}
// (a, b) * (c, d).
__device__ __forceinline__ float2 mul2(float2 a, float2 b) {
  float2 o;
  asm("{\n .reg .b64 x, y, z;\n mov.b64 x, {%2, %3};\n mov.b64 y, {%4, %5};\n mul.rn.f32x2 z, x, y;\n"
      " mov.b64 {%0, %1}, z;\n}"
      : "=f"(o.x), "=f"(o.y)
      : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y));
  return o;
}
// x silu(g) of two elements. Units of 2^-24: the exponent 1.25 |g| (its product, log2 e),
// ex2 4, 1 + e 1, the reciprocal 2, two products: 1.25 |g| + 9. (x by the reciprocal first:
// half a gate below the normal numbers would lose bits that a large x makes count. Where x by
// the reciprocal is below them, either the reciprocal is 1 or y is too small for any code.)
__device__ __forceinline__ float2 gated(float2 x, float2 g) {
  const float2 t = mul2(g.x, g.y, -1.4426950408889634f);
  const float2 e = plus1(make_float2(ex2_approx(t.x), ex2_approx(t.y)));
  return mul2(mul2(x, make_float2(rcp_approx(e.x), rcp_approx(e.y))), g);
}

// Which code is that of y, `code` or the next one away from zero: that of the nearer
// value, num |y| - m den deciding on their border m.
__device__ __forceinline__ uint32_t nearer(uint32_t code, Wide y, float num, Wide den) {
  const uint32_t sign = code & 0x80u, lower = code & 0x7Fu;
  uint32_t two;  // the codes' values
  asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(two) : "h"(uint16_t(lower | ((lower + 1) << 8))));
  const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&two));
  const float m = 0.5f * (f.x + f.y);
  // (large numbers are made smaller, by a power of two: 448 y is at most fp32's largest)
  const float k = den.hi > 0x1p100f ? 0x1p-32f : 1.f;
  const float yh = fabsf(y.hi) * k, yl = (y.hi < 0.f ? -y.lo : y.lo) * k, dh = den.hi * k, dl = den.lo * k;
  const float v = num * yh, w = m * dh;
  const float over = (v - w) + ((__fmaf_rn(num, yh, -v) - __fmaf_rn(m, dh, -w)) + (num * yl - m * dl));
  return sign | (over > 0.f ? lower + 1 : over < 0.f ? lower : lower + (lower & 1));
}

// A lane's sixteen elements of a group, two runs of eight, and what is done to them.
template <typename T, int kMode>
struct Item {
  static constexpr bool kTurns = kMode == kAdjacent || kMode == kHalves;

  Eight<T> x[2], gate[2];
  int row;      // output row, -1: nothing is stored
  int k0;       // the lane's first element in the row; the other run is 64 further
  int r, pos;   // kTurns: the first element's place in the rotated range, the row's position
  bool live[2];

  // The lane's part of the group of row `out` (out >= p.rows: of none) that begins at
  // element d of head row h, element k of the row.
  __device__ __forceinline__ void load(const qsfm_quantize_params& p, const QuantizeShape& s, uint32_t out, uint32_t h,
                                       int d, int k, int* fault) {
    const int sub = threadIdx.x & (kQLanes - 1);
    row = out < uint32_t(p.rows) ? int(out) : -1;
    k0 = k + 8 * sub;
    d += 8 * sub;
    int src = row;
    if (p.row_index != nullptr && row >= 0) {
      src = __ldg(p.row_index + row);
      if (src < 0 || src >= p.source_rows) {
        if (src >= 0 && sub == 0) atomicOr(fault, QSFM_FAULT_ROW_INDEX);
        row = -1;
      }
    }
    pos = 0;
    if (p.positions != nullptr && row >= 0) pos = __ldg(p.positions + row);  // looked at in check()
    const T* from = static_cast<const T*>(p.x) + size_t(src) * p.x_row_stride + size_t(h) * p.x_head_stride + d;
    const T* with = static_cast<const T*>(p.gate) + size_t(src) * p.gate_row_stride + size_t(h) * p.gate_head_stride + d;
#pragma unroll
    for (int j = 0; j < 2; ++j) {
      live[j] = row >= 0 && k0 + 64 * j < s.k;
      if (live[j]) {
        x[j].load(from + 64 * j);
        if constexpr (kMode == kGated) gate[j].load(with + 64 * j);
      } else {
        x[j].zero();
        if constexpr (kMode == kGated) gate[j].zero();
      }
    }
    if constexpr (kTurns) r = d - p.rope_offset;
  }

  // Drops the row where its position says so (after all loads are on their way).
  __device__ __forceinline__ void check(const qsfm_quantize_params& p, int* fault) {
    if (pos < 0 || (p.rope_dim > 0 && row >= 0 && pos >= p.max_positions)) {
      if (pos >= 0 && (threadIdx.x & (kQLanes - 1)) == 0) atomicOr(fault, QSFM_FAULT_POSITION);
      row = -1;
      live[0] = live[1] = false;
    }
  }

  // Whether run j is turned.
  __device__ __forceinline__ bool in(const qsfm_quantize_params& p, int j) const {
    return kTurns && live[j] && r + 64 * j >= 0 && r + 64 * j < p.rope_dim;
  }

  // Cosines and sines of run j (a position's row of the table serves all heads of its
  // token, so it comes from the caches), the sines with the sign that makes an element
  // a c - b s; of adjacent pairs four of each.
  __device__ __forceinline__ void load_angles(const qsfm_quantize_params& p, int j, float (&c)[8], float (&s)[8]) const {
    const int half = p.rope_dim / 2, at = r + 64 * j;
    const float* from = p.cos_sin + size_t(pos) * p.rope_dim + (kMode == kAdjacent ? at / 2 : at >= half ? at - half : at);
#pragma unroll
    for (int i = 0; i < (kMode == kAdjacent ? 4 : 8); i += 4) {
      const float4 a = __ldg(reinterpret_cast<const float4*>(from + i));
      const float4 b = __ldg(reinterpret_cast<const float4*>(from + half + i));
      c[i] = a.x; c[i + 1] = a.y; c[i + 2] = a.z; c[i + 3] = a.w;
      s[i] = b.x; s[i + 1] = b.y; s[i + 2] = b.z; s[i + 3] = b.w;
    }
    const bool flip = (p.inverse != 0) != (kMode == kHalves && at >= half);
#pragma unroll
    for (int i = 0; i < (kMode == kAdjacent ? 4 : 8); ++i) s[i] = flip ? -s[i] : s[i];
  }

  // The elements y. kGated: `large` becomes whether one of the warp's gates is above 12
  // in magnitude.
  template <int kAs>
  __device__ __forceinline__ void values(const qsfm_quantize_params& p, float (&y)[kQElems], bool& large) const {
    x[0].get(y);
    x[1].get(y + 8);
    if constexpr (kMode == kGated) {
      float top = 0.f;
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        float g[8];
        gate[j].get(g);
#pragma unroll
        for (int i = 0; i < 8; i += 2) {
          top = abs_max(top, g[i]);
          top = abs_max(top, g[i + 1]);
          const float2 v = gated(make_float2(y[8 * j + i], y[8 * j + i + 1]), make_float2(g[i], g[i + 1]));
          y[8 * j + i] = v.x;
          y[8 * j + i + 1] = v.y;
        }
      }
      large = __any_sync(kAllLanes, !(top <= 12.f));
    }
    if constexpr (kTurns && kAs != kPlain) {
      float z[kQElems];  // the inputs (both runs are turned from them)
#pragma unroll
      for (int i = 0; i < kQElems; ++i) z[i] = y[i];
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        if (!__any_sync(kAllLanes, in(p, j))) continue;
        float other[8];  // what an element is turned with
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          if constexpr (kMode == kAdjacent) other[i] = z[8 * j + (i ^ 1)];
          else if (p.rope_dim == 128) other[i] = z[8 * (j ^ 1) + i];
          else other[i] = __shfl_xor_sync(kAllLanes, z[8 * j + i], p.rope_dim / 16);
        }
        if (!in(p, j)) continue;
        float c[8], s[8];
        load_angles(p, j, c, s);
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          const int k = kMode == kAdjacent ? i / 2 : i;
          y[8 * j + i] = turned(z[8 * j + i], c[k], other[i], kMode == kAdjacent && (i & 1) ? -s[k] : s[k]);
        }
      }
    }
  }
};

// Whether y, as far as its fp32 value may be off, can be the group's largest, which is m in
// fp32: 256 units of difference are more than the errors of both (118 units of 2^-24 at most).
__device__ __forceinline__ bool may_be_top(float y, float m) {
  return (__float_as_uint(y) & 0x7FFFFFFFu) + 256u >= __float_as_uint(m);
}

// The largest |y| of the lane's runs and of the group, NaN when one is.
__device__ __forceinline__ float group_max(const float (&y)[kQElems], float (&run)[2]) {
#pragma unroll
  for (int j = 0; j < 2; ++j) {
    run[j] = abs_max(y[8 * j], y[8 * j + 1]);
#pragma unroll
    for (int i = 2; i < 8; ++i) run[j] = abs_max(run[j], y[8 * j + i]);
  }
  float m = abs_max(run[0], run[1]);
#pragma unroll
  for (int o = kQLanes / 2; o > 0; o >>= 1) m = abs_max(m, __shfl_xor_sync(kAllLanes, m, o));
  return m;
}

// Element i (0 .. 15) of the lane whose first is k0 of output row `row`, from memory, as
// a sum of two fp32 values.
template <typename T, int kMode>
__device__ __forceinline__ Wide wide_element(const qsfm_quantize_params& p, int row, int k0, int i) {
  const int k = k0 + (i & 7) + (i >= 8 ? 64 : 0);
  const int h = p.heads > 1 ? k / p.dim : 0, d = k - h * p.dim;
  const size_t src = size_t(p.row_index != nullptr ? __ldg(p.row_index + row) : row);
  const T* x = static_cast<const T*>(p.x) + src * p.x_row_stride + size_t(h) * p.x_head_stride;
  const float v = float(x[d]);
  if constexpr (kMode == kGated) {
    const double g = float(static_cast<const T*>(p.gate)[src * p.gate_row_stride + size_t(h) * p.gate_head_stride + d]);
    const double y = double(v) * (g / (1.0 + exp(-g)));
    const float hi = float(y);
    return {hi, float(y - double(hi))};
  }
  const int r = d - p.rope_offset;
  if ((kMode == kAdjacent || kMode == kHalves) && r >= 0 && r < p.rope_dim) {
    const int half = p.rope_dim / 2;
    const bool second = kMode == kAdjacent ? (r & 1) != 0 : r >= half;
    const int pair = kMode == kAdjacent ? r / 2 : second ? r - half : r;
    const int apart = kMode == kAdjacent ? 1 : half;
    const float* c = p.cos_sin + size_t(__ldg(p.positions + row)) * p.rope_dim + pair;
    const float s = (p.inverse != 0) != second ? -c[half] : c[half];
    return turned_wide(v, c[0], float(x[second ? d - apart : d + apart]), s);
  }
  return {v, 0.f};
}

// The elements of a lane that may hold the group's largest |y|, which is m in fp32.
__device__ __forceinline__ uint32_t near_top(const float (&y)[kQElems], float m) {
  uint32_t which = 0;
#pragma unroll
  for (int i = 0; i < kQElems; ++i)
    which |= may_be_top(y[i], m) ? 1u << i : 0u;
  return which;
}

// The largest |y| of the group among the elements that `which` has a bit for. The whole
// warp calls it. (Out of line, as fix_borders(): a loop over single elements from memory,
// so that a path that one warp in a hundred takes costs the others no registers and
// little of the instruction cache.)
template <typename T, int kMode>
__device__ __noinline__ float2 wide_top(const qsfm_quantize_params& p, int row, int k0, uint32_t which) {
  Wide top = {0.f, 0.f};
  for (; which != 0; which &= which - 1) {
    Wide v = wide_element<T, kMode>(p, row, k0, __ffs(which) - 1);
    if (v.hi < 0.f) v = {-v.hi, -v.lo};
    if (v.hi > top.hi || (v.hi == top.hi && v.lo > top.lo)) top = v;
  }
  __syncwarp();
#pragma unroll
  for (int o = kQLanes / 2; o > 0; o >>= 1) {
    const Wide v = {__shfl_xor_sync(kAllLanes, top.hi, o), __shfl_xor_sync(kAllLanes, top.lo, o)};
    if (v.hi > top.hi || (v.hi == top.hi && v.lo > top.lo)) top = v;
  }
  return make_float2(top.hi, top.lo);
}

// Stores the codes of the lane's elements that `which` has a bit for, each one of two
// neighbours, the lower of which (without its sign) is already stored.
template <typename T, int kMode>
__device__ __noinline__ void fix_borders(const qsfm_quantize_params& p, int row, int k0, uint32_t which, float num,
                                         Wide den) {
  uint8_t* codes = static_cast<uint8_t*>(p.codes) + size_t(row) * (size_t(p.heads) * p.dim) + k0;
  for (; which != 0; which &= which - 1) {
    const int i = __ffs(which) - 1;
    uint8_t* at = codes + (i & 7) + (i >= 8 ? 64 : 0);
    *at = uint8_t(nearer(*at, wide_element<T, kMode>(p, row, k0, i), num, den));
  }
}

// A lane's codes of an item, and its group's scale. kMode is kPlain for items of which
// nothing is turned, whatever they were loaded as.
template <typename T, int kMode, typename I>
__device__ __forceinline__ void finish(const qsfm_quantize_params& p, const QuantizeShape& s, const I& item,
                                       size_t scale_at) {
  constexpr bool kTurns = kMode == kAdjacent || kMode == kHalves;
  float y[kQElems], run[2];
  bool large = false;
  item.template values<kMode>(p, y, large);
  // At least the relative error of a quotient, in units of 2^-24: those of y (turned 3,
  // gated 24 up to a gate of 12 and 118 up to 87), r (1 -+ error) 1; without powers of two
  // also those of A (as many as of y), r 3, the product y r 1.
  float error = kTurns ? 0x1p-20f : 0x1p-21f;
  if constexpr (kMode == kGated) error = p.pow2_scale ? (large ? 0x1p-17f : 0x1p-19f) : (large ? 0x1p-16f : 0x1p-18f);
  const uint32_t own = (item.live[0] ? 0xFFu : 0u) | (item.live[1] ? 0xFF00u : 0u);  // the lane's elements in the row
  constexpr bool computed = kMode != kPlain;
  const float m = group_max(y, run);
  const bool bad = !(m < __uint_as_float(0x7F800000u));  // an element is not finite
  const float a = fmaxf(bad ? 1.f : m, kQMin);
  float scale, r;
  uint32_t c[4];
  if (p.pow2_scale) {
    int e = pow2_exponent(m);
    if (computed) {
      // A next to 1.75 2^j, where e changes
      const bool near = !bad && abs(int(__float_as_uint(m) & 0x7FFFFFu) - 0x600000) < 128;
      if (__any_sync(kAllLanes, near)) {
        const float2 top = wide_top<T, kMode>(p, item.row, item.k0, near ? near_top(y, m) & own : 0);
        if (near) e = pow2_exponent(top.x, top.y);
      }
    }
    scale = power2(e);
    r = power2(-e);
    if (!computed) codes16<false>(y, r, c);  // exact
  } else {
    scale = over448(a);
    r = 0.875f * rcp_approx(a * 0x1p-9f);  // 448 / a; 512 / a is normal for every a
    if constexpr (sizeof(T) == 2 && kMode != kGated) codes16<true>(y, r * (1.f + 0x1.8p-22f), c);
  }
  // the elements that lie next to a border by chance: those that are not an input over an input
  uint32_t which = 0;
  if (computed || (sizeof(T) == 4 && !p.pow2_scale)) {
    uint32_t chance = 0xFFFFu;
    if constexpr (kTurns) {
      if (sizeof(T) == 2 || p.pow2_scale) {
        // A is computed where a lane of the group may hold it among its turned elements
        // (one whose fp32 value is below m may itself be above)
        const bool holds = (item.in(p, 0) && may_be_top(run[0], m)) || (item.in(p, 1) && may_be_top(run[1], m));
        const bool of_group = !p.pow2_scale && (__ballot_sync(kAllLanes, holds) >> (threadIdx.x & 24u) & 0xFFu) != 0;
        chance = of_group ? 0xFFFFu : (item.in(p, 0) ? 0xFFu : 0u) | (item.in(p, 1) ? 0xFF00u : 0u);
      }
    }
    uint32_t lo[4], hi[4];
    codes16<false>(y, r * (1.f - error), lo);
    codes16<false>(y, r * (1.f + error), hi);
    const bool plain[2] = {(chance & 1) == 0, (chance & 0x100u) == 0};
    if constexpr (kTurns) {
      if (p.pow2_scale && (plain[0] || plain[1])) {
        uint32_t exact[4];
        codes16<false>(y, r, exact);
#pragma unroll
        for (int i = 0; i < 4; ++i) c[i] = exact[i];
      }
    }
    bool differ = false;
#pragma unroll
    for (int i = 0; i < 4; ++i)
      if (!plain[i / 2]) {
        c[i] = lo[i];
        differ = differ || lo[i] != hi[i];
      }
    if (__any_sync(kAllLanes, differ && !bad)) {
#pragma unroll
      for (int i = 0; i < kQElems; ++i)
        which |= ((lo[i / 4] ^ hi[i / 4]) >> (8 * (i & 3)) & 0xFFu) != 0 ? chance & (1u << i) : 0u;
      if (bad) which = 0;
    }
  }
  if (bad) {
    scale = __uint_as_float(0x7FC00000u);
#pragma unroll
    for (int i = 0; i < 4; ++i) c[i] = 0x7F7F7F7Fu;
  }
  uint8_t* to = static_cast<uint8_t*>(p.codes) + size_t(uint32_t(item.row)) * s.k + item.k0;
  if (item.live[0]) *reinterpret_cast<uint2*>(to) = make_uint2(c[0], c[1]);
  if (item.live[1]) *reinterpret_cast<uint2*>(to + 64) = make_uint2(c[2], c[3]);
  if (item.row >= 0 && (threadIdx.x & (kQLanes - 1)) == 0) p.scale[scale_at] = scale;
  if (kMode != kPlain || sizeof(T) == 4) {
    which &= own;
    if (__any_sync(kAllLanes, which != 0)) {
      Wide den = {a, a == kQMin ? kQMinRest : 0.f};
      if (p.pow2_scale) {
        den = {scale, 0.f};
      } else if (kMode != kPlain) {
        const float2 top = wide_top<T, kMode>(p, item.row, item.k0, bad ? 0 : near_top(y, m) & own);
        const bool least = top.x < kQMin || (top.x == kQMin && top.y <= kQMinRest);
        den = least ? Wide{kQMin, kQMinRest} : Wide{top.x, top.y};
      }
      if (which != 0) fix_borders<T, kMode>(p, item.row, item.k0, which, p.pow2_scale ? 1.f : 448.f, den);
      __syncwarp();
    }
  }
}

// kItems times four groups per warp: neighbours in a row or, where a part of each head is
// turned (kHeads), the same group of four heads in a row, so that what is turned is in
// warps of its own.
template <typename T, int kMode, int kItems, bool kHeads>
__global__ void __launch_bounds__(32 * kQWarps, blocks_per_sm(kMode))
    quantize_kernel(const __grid_constant__ qsfm_quantize_params p, const __grid_constant__ QuantizeShape s, int* fault) {
  grid_dependency_wait();
  grid_launch_dependents();
  const uint32_t quarter = (threadIdx.x & 31) >> 3;
  const uint32_t first = (blockIdx.x * kQWarps + (threadIdx.x >> 5)) * kItems;
  if (first >= s.units) return;  // the whole warp
  Item<T, kMode> item[kItems];
  size_t scale_at[kItems];
#pragma unroll
  for (int u = 0; u < kItems; ++u) {
    if constexpr (kHeads) {
      const uint32_t four = s.groups_of.div(first + u), head = 4 * four + quarter, row = s.heads_of.div(head);
      const uint32_t h = head - row * uint32_t(p.heads);
      uint32_t g = first + u - four * s.groups_of.d + s.first;
      if (g >= s.skip) ++g;
      scale_at[u] = size_t(head) * s.of_head + g;
      item[u].load(p, s, first + u < s.units ? row : 0xffffffffu, h, int(g) * kQGroup, int(h) * p.dim + int(g) * kQGroup, fault);
    } else {
      const uint32_t f = 4 * (first + u) + quarter, row = s.groups_of.div(f), g = f - row * s.groups_of.d;
      const uint32_t h = p.heads > 1 ? s.heads_of.div(g) : 0;
      scale_at[u] = f;
      item[u].load(p, s, row, h, int(g) * kQGroup - int(h) * p.dim, int(g) * kQGroup, fault);
    }
  }
#pragma unroll
  for (int u = 0; u < kItems; ++u) {
    item[u].check(p, fault);
    if (Item<T, kMode>::kTurns && !__any_sync(kAllLanes, item[u].in(p, 0) || item[u].in(p, 1)))
      finish<T, kPlain>(p, s, item[u], scale_at[u]);
    else
      finish<T, kMode>(p, s, item[u], scale_at[u]);
  }
}

template <typename T, int kMode, int kItems, bool kHeads>
cudaError_t launch_units(const qsfm_quantize_params& p, const QuantizeShape& s, int* fault, cudaStream_t stream) {
  const uint32_t warps = (s.units + kItems - 1) / kItems;
  return launch_after_predecessor(quantize_kernel<T, kMode, kItems, kHeads>, dim3((warps + kQWarps - 1) / kQWarps),
                                  dim3(32 * kQWarps), 0, stream, p, s, fault);
}

// Units of four groups up to which a warp takes one, so that they spread over the SMs (of a
// GB300, 32 warps each); with more it has 64 bytes of the inputs a lane on their way.
constexpr uint32_t kFewUnits = 152 * 32;

template <typename T, int kMode>
cudaError_t launch_mode(const qsfm_quantize_params& p, int* fault, cudaStream_t stream) {
  constexpr int kItems = sizeof(T) == 4 || kMode == kGated ? 1 : 2;
  QuantizeShape s;
  s.k = p.heads * p.dim;
  const uint32_t groups = uint32_t((s.k + kQGroup - 1) / kQGroup);
  s.of_head = uint32_t((p.dim + kQGroup - 1) / kQGroup);
  s.first = 0;
  s.skip = 0xffffffffu;
  if constexpr (Item<T, kMode>::kTurns) {
    const uint32_t fours = uint32_t((uint64_t(p.rows) * uint32_t(p.heads) + 3) / 4);
    s.heads_of.set(uint32_t(p.heads));
    s.groups_of.set(s.of_head);
    s.units = fours * s.of_head;
    if (s.units <= kFewUnits) return launch_units<T, kMode, 1, true>(p, s, fault, stream);
    // of many, the groups that nothing is turned of in a launch of the kernel for them,
    // which has twice the warps on an SM (4099 tokens of 64 heads: 91 us in one launch)
    const uint32_t turned = uint32_t(p.rope_offset) / kQGroup;
    if (s.of_head > 1) {
      QuantizeShape rest = s;
      rest.groups_of.set(s.of_head - 1);
      rest.units = fours * (s.of_head - 1);
      rest.skip = turned;
      const cudaError_t e = launch_units<T, kPlain, kItems, true>(p, rest, fault, stream);
      if (e != cudaSuccess) return e;
    }
    s.groups_of.set(1);
    s.units = fours;
    s.first = turned;
    return launch_units<T, kMode, kItems, true>(p, s, fault, stream);
  } else {
    s.groups_of.set(groups);
    s.heads_of.set(s.of_head);
    s.units = (uint32_t(p.rows) * groups + 3) / 4;
    if (kItems == 1 || s.units <= kFewUnits) return launch_units<T, kMode, 1, false>(p, s, fault, stream);
    return launch_units<T, kMode, kItems, false>(p, s, fault, stream);
  }
}

template <typename T>
cudaError_t launch_type(const qsfm_quantize_params& p, int* fault, cudaStream_t stream) {
  if (p.gate != nullptr) return launch_mode<T, kGated>(p, fault, stream);
  if (p.rope_dim > 0 && p.interleaved) return launch_mode<T, kAdjacent>(p, fault, stream);
  if (p.rope_dim > 0) return launch_mode<T, kHalves>(p, fault, stream);
  return launch_mode<T, kPlain>(p, fault, stream);
}

}  // namespace

cudaError_t launch_quantize(const qsfm_quantize_params& p, int* fault, cudaStream_t stream) {
  switch (p.in_type) {
    case QSFM_BF16: return launch_type<__nv_bfloat16>(p, fault, stream);
    case QSFM_F16: return launch_type<__half>(p, fault, stream);
    default: return launch_type<float>(p, fault, stream);
  }
}

}  // namespace qsfm
