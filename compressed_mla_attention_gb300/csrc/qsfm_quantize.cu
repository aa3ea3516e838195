// Rows quantised to e4m3 with one fp32 scale per 128 elements (sm_103a).
//
// For each group of 128 elements y of a row, with A = max|y| (at least 1e-12):
//   scale = A / 448, code = e4m3(448 y / A) to nearest even, or, with scales that
//   are powers of two, scale = 2^e of the smallest e with A <= 448 2^e.
// y is the input itself, the input times silu(gate), or the input with a part of
// each head turned by its position's angles; a row may be taken from anywhere in
// the input (row_index).
//
// Sixteen lanes hold a group, eight neighbouring elements each, so A is four
// shuffles of a maximum over the elements' bits (which also carries an inf or NaN
// through), a pair of the rotation is in the lane (adjacent) or rope_dim / 16 lanes
// apart (halves), and a group's codes are one 128-byte line. The kernel is bound by
// HBM: a warp has the loads of 2 kItems groups in flight.
//
// Every code is the formula's. The fast path rounds 448 y / A with an error e of a
// few units of fp32, so it converts the quotient twice, times 1 - e and 1 + e: where
// both give the same code, that is the code. Elsewhere (an element next to the border
// of two codes) the quotient is made again: for 16-bit inputs by a division, whose
// fp32 result cannot cross a border (x has 8 or 11 significant bits, A as many and a
// border five, so that 448 x and border * A are either equal or 2^-17 apart); for
// computed y, and fp32 inputs, in 64 bits.
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include <type_traits>

#include "qsfm_device.cuh"
#include "qsfm_internal.h"

namespace qsfm {
namespace {

constexpr int kQGroup = 128;                 // elements of a scale
constexpr int kQWarps = 8;
constexpr uint32_t kAllLanes = 0xffffffffu;
constexpr float kQMin = 1e-12f;              // A of an all-zero group

enum QuantizeMode { kPlain = 0, kRotate = 1, kGated = 2 };

// Division of 31-bit numbers by an invariant d: q = (n * m) >> (32 + s) with
// m = ceil(2^(32 + s) / d), s = ceil(log2 d) - 1 (exact for n < 2^31).
struct FastDiv {
  uint32_t d, m, s;
  __host__ void set(uint32_t div) {
    d = div;
    s = 0;
    while ((2u << s) < div) ++s;
    m = div <= 1 ? 0 : uint32_t(((1ull << (32 + s)) + div - 1) / div);
  }
  __device__ __forceinline__ uint32_t div(uint32_t n) const { return d <= 1 ? n : __umulhi(n, m) >> s; }
};

struct QuantizeShape {
  uint32_t groups;   // scales of a row
  uint32_t total;    // rows * groups
  int k;             // elements of a row
  FastDiv per_row;   // by groups
  FastDiv per_head;  // by the groups of a head row
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
  __device__ __forceinline__ void get(float (&f)[8]) const {
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

// e4m3 codes of a (low byte) and b, to nearest even, saturating.
__device__ __forceinline__ uint32_t e4m3x2(float a, float b) {
  uint16_t r;
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(r) : "f"(b), "f"(a));
  return r;
}
__device__ __forceinline__ uint2 codes8(const float (&q)[8], float r) {
  return make_uint2(e4m3x2(q[0] * r, q[1] * r) | (e4m3x2(q[2] * r, q[3] * r) << 16),
                    e4m3x2(q[4] * r, q[5] * r) | (e4m3x2(q[6] * r, q[7] * r) << 16));
}

// fp64 to fp32, a result that is not exact made odd: a rounding to fewer bits that
// follows is then that of the fp64 value.
__device__ __forceinline__ float round_odd(double x) {
  const float f = __double2float_rz(x);
  return double(f) == x ? f : __uint_as_float(__float_as_uint(f) | 1u);
}

// The smallest e with a <= 448 2^e = 1.75 2^(8 + e), within -100 .. 100.
__device__ __forceinline__ int pow2_exponent(float a) {
  const uint32_t u = __float_as_uint(a);
  return min(max(int(u >> 23) - 127 - 8 + ((u & 0x7FFFFFu) > 0x600000u ? 1 : 0), -100), 100);
}
__device__ __forceinline__ int pow2_exponent(double a) {
  const uint64_t u = uint64_t(__double_as_longlong(a));
  return min(max(int(u >> 52) - 1023 - 8 + ((u & 0xFFFFFFFFFFFFFull) > 0xC000000000000ull ? 1 : 0), -100), 100);
}
__device__ __forceinline__ float power2(int e) { return __uint_as_float(uint32_t(e + 127) << 23); }

// The lane's cosines and sines: adjacent pairs use four of each, halves eight.
struct Angles {
  float c[8], s[8];
};

// y = x turned: lanes with `in` hold elements of the rotated range. The products'
// difference with what its roundings leave over (each result within 1.5 units), so
// that y is as good where its terms cancel.
__device__ __forceinline__ float turned(float a, float c, float b, float s) {  // a c - b s
  const float w = b * s;
  return __fmaf_rn(a, c, -w) + __fmaf_rn(-b, s, w);
}
template <typename V>
__device__ __forceinline__ V turned(V a, V c, V b, V s) {
  return a * c - b * s;
}
template <typename V>
__device__ __forceinline__ void turn(const qsfm_quantize_params& p, bool in, int r, const Angles& t, V (&y)[8]) {
  if (p.interleaved) {
    if (in) {
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const V a = y[2 * i], b = y[2 * i + 1];
        y[2 * i] = turned(a, V(t.c[i]), b, V(t.s[i]));
        y[2 * i + 1] = turned(b, V(t.c[i]), a, V(-t.s[i]));
      }
    }
  } else {
    const int apart = p.rope_dim / 16;  // lanes between the elements of a pair
    const bool second = r >= p.rope_dim / 2;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const V other = __shfl_xor_sync(kAllLanes, y[i], apart);
      if (in) y[i] = turned(y[i], V(t.c[i]), other, V(second ? -t.s[i] : t.s[i]));
    }
  }
}

__device__ __forceinline__ float silu(float g) { return g * __fdividef(1.f, 1.f + expf(-g)); }
__device__ __forceinline__ double silu(double g) { return g / (1.0 + exp(-g)); }

// One item of a lane: eight elements of group f and what they are multiplied by.
template <typename T, int kMode>
struct Item {
  Eight<T> x, gate;
  int row;       // output row, -1: nothing is stored
  int k0;        // the lane's first element in the row
  int r, pos;    // kRotate: its place in the rotated range, the row's position
  bool live, in;

  __device__ __forceinline__ void load(const qsfm_quantize_params& p, const QuantizeShape& s, uint32_t f, int sub,
                                       int* fault) {
    live = f < s.total;
    const uint32_t out = s.per_row.div(f), g = f - out * s.groups;
    row = live ? int(out) : -1;
    k0 = int(g) * kQGroup + 8 * sub;
    live = live && k0 < s.k;
    int src = row;
    if (p.row_index != nullptr && row >= 0) {
      src = __ldg(p.row_index + row);
      if (src < 0 || src >= p.source_rows) {
        if (src >= 0 && sub == 0) atomicOr(fault, QSFM_FAULT_ROW_INDEX);
        row = -1;
      }
    }
    pos = 0;
    if (p.positions != nullptr && row >= 0) {
      pos = __ldg(p.positions + row);
      if (pos < 0 || (kMode == kRotate && pos >= p.max_positions)) {
        if (pos >= 0 && sub == 0) atomicOr(fault, QSFM_FAULT_POSITION);
        row = -1;
      }
    }
    live = live && row >= 0;
    const uint32_t h = p.heads > 1 ? s.per_head.div(g) : 0;
    const int d = k0 - int(h) * p.dim;  // element of the head row
    if (live) {
      x.load(static_cast<const T*>(p.x) + size_t(src) * p.x_row_stride + size_t(h) * p.x_head_stride + d);
      if constexpr (kMode == kGated)
        gate.load(static_cast<const T*>(p.gate) + size_t(src) * p.gate_row_stride + size_t(h) * p.gate_head_stride + d);
    } else {
      x.zero();
      if constexpr (kMode == kGated) gate.zero();
    }
    if constexpr (kMode == kRotate) {
      r = d - p.rope_offset;
      in = live && r >= 0 && r < p.rope_dim;
    }
  }

  // The angles of the lane's pairs (a position's row of the table serves all heads of
  // its token, so it comes from the caches; held from the load on, the angles of four
  // items would cost 64 registers).
  __device__ __forceinline__ void load_angles(const qsfm_quantize_params& p, Angles& t) const {
    if (!in) return;
    const int half = p.rope_dim / 2, at = p.interleaved ? r / 2 : r >= half ? r - half : r;
    const float* c = p.cos_sin + size_t(pos) * p.rope_dim + at;
#pragma unroll
    for (int i = 0; i < 8; i += 4) {
      if (i > 0 && p.interleaved) break;
      const float4 a = __ldg(reinterpret_cast<const float4*>(c + i));
      const float4 b = __ldg(reinterpret_cast<const float4*>(c + half + i));
      t.c[i] = a.x; t.c[i + 1] = a.y; t.c[i + 2] = a.z; t.c[i + 3] = a.w;
      t.s[i] = b.x; t.s[i + 1] = b.y; t.s[i + 2] = b.z; t.s[i + 3] = b.w;
    }
    if (p.inverse) {
#pragma unroll
      for (int i = 0; i < 8; ++i) t.s[i] = -t.s[i];
    }
  }

  template <typename V>
  __device__ __forceinline__ void values(const qsfm_quantize_params& p, const Angles& t, V (&y)[8]) const {
    float f[8];
    x.get(f);
#pragma unroll
    for (int i = 0; i < 8; ++i) y[i] = V(f[i]);
    if constexpr (kMode == kGated) {
      gate.get(f);
#pragma unroll
      for (int i = 0; i < 8; ++i) y[i] *= silu(V(f[i]));
    }
    if constexpr (kMode == kRotate) turn(p, in, r, t, y);
  }

  // The codes of the lane's elements and the group's scale.
  __device__ __forceinline__ uint2 codes(const qsfm_quantize_params& p, float& scale) const {
    float y[8];
    Angles t;
    if constexpr (kMode == kRotate) load_angles(p, t);
    values(p, t, y);
    uint32_t m = 0;
#pragma unroll
    for (int i = 0; i < 8; ++i) m = max(m, __float_as_uint(y[i]) & 0x7FFFFFFFu);
#pragma unroll
    for (int o = 8; o > 0; o >>= 1) m = max(m, __shfl_xor_sync(kAllLanes, m, o));
    const bool bad = m >= 0x7F800000u;  // an element is not finite
    const float top32 = bad ? 1.f : __uint_as_float(m), a = fmaxf(top32, kQMin);
    // at least the relative error of a quotient, in units of 2^-24: those of y (kRotate
    // 3; kGated 9: expf 2, 1 + e 1, the division 4, two products), those of A (as
    // many), r 1, the products r (1 +- kErr) and y r 2
    constexpr float kErr = kMode == kGated ? 0x1p-19f : kMode == kRotate ? 0x1p-20f : 0x1p-21f;
    float r;
    bool near_power = false;
    if (p.pow2_scale) {
      const int e = pow2_exponent(top32);
      scale = power2(e);
      r = power2(-e);
      if constexpr (kMode != kPlain) near_power = abs(int(__float_as_uint(top32) & 0x7FFFFFu) - 0x600000) < 64;
    } else {
      r = __fdiv_rn(448.f, a);
      scale = __fdiv_rn(a, 448.f);
    }
    uint2 c = codes8(y, r * (1.f - kErr));
    const uint2 d = codes8(y, r * (1.f + kErr));
    const bool differ = c.x != d.x || c.y != d.y;
    if constexpr (kMode == kPlain) {
      if (differ) {
        if constexpr (sizeof(T) == 2) {
          if (p.pow2_scale) {
            c = codes8(y, r);  // exact
          } else {
            float q[8];
#pragma unroll
            for (int i = 0; i < 8; ++i) q[i] = __fdiv_rn(y[i] * 0.4375f, a);  // 448 / 1024: no overflow
            c = codes8(q, 1024.f);
          }
        } else {
          float q[8];
#pragma unroll
          for (int i = 0; i < 8; ++i) q[i] = p.pow2_scale ? y[i] * r : round_odd(double(y[i]) * 448.0 / double(a));
          c = codes8(q, 1.f);
        }
      }
    } else {
      // the warp's two groups again where one has such an element: the branch holds shuffles
      if (__any_sync(kAllLanes, (differ || near_power) && !bad)) {
        double z[8], top = 0.0;
        values(p, t, z);
#pragma unroll
        for (int i = 0; i < 8; ++i) top = fmax(top, fabs(z[i]));
#pragma unroll
        for (int o = 8; o > 0; o >>= 1) top = fmax(top, __shfl_xor_sync(kAllLanes, top, o));
        const int e = pow2_exponent(top);
        top = fmax(top, double(kQMin));
        float q[8];
        if (p.pow2_scale) {
          scale = power2(e);
          const double step = double(power2(-e));
#pragma unroll
          for (int i = 0; i < 8; ++i) q[i] = round_odd(z[i] * step);
        } else {
          scale = float(top / 448.0);
#pragma unroll
          for (int i = 0; i < 8; ++i) q[i] = round_odd(z[i] * 448.0 / top);
        }
        c = codes8(q, 1.f);
      }
    }
    if (bad) {
      scale = __uint_as_float(0x7FC00000u);
      c = make_uint2(0x7F7F7F7Fu, 0x7F7F7F7Fu);
    }
    return c;
  }
};

// kItems pairs of neighbouring groups per warp: half a warp a group.
template <typename T, int kMode, int kItems>
__global__ void __launch_bounds__(32 * kQWarps)
    quantize_kernel(const qsfm_quantize_params p, const QuantizeShape s, int* fault) {
  grid_dependency_wait();
  grid_launch_dependents();
  const int lane = threadIdx.x & 31, half = lane >> 4, sub = lane & 15;
  const uint32_t warp = blockIdx.x * kQWarps + (threadIdx.x >> 5);
  const uint32_t first = warp * (2 * kItems);
  if (first >= s.total) return;  // the whole warp
  Item<T, kMode> item[kItems];
#pragma unroll
  for (int u = 0; u < kItems; ++u) item[u].load(p, s, first + 2 * u + half, sub, fault);
#pragma unroll
  for (int u = 0; u < kItems; ++u) {
    float scale;
    const uint2 c = item[u].codes(p, scale);
    if (item[u].live)
      *reinterpret_cast<uint2*>(static_cast<uint8_t*>(p.codes) + size_t(item[u].row) * s.k + item[u].k0) = c;
    if (item[u].row >= 0 && sub == 0) p.scale[first + 2 * u + half] = scale;
  }
}

template <typename T, int kMode>
cudaError_t launch_mode(const qsfm_quantize_params& p, const QuantizeShape& s, int* fault, cudaStream_t stream) {
  // few groups: one pair a warp, so that they spread over the SMs; many: four, for
  // the bytes in flight
  const uint32_t pairs = (s.total + 1) / 2;
  if (pairs <= 152 * 32) {
    return launch_after_predecessor(quantize_kernel<T, kMode, 1>, dim3((pairs + kQWarps - 1) / kQWarps),
                                    dim3(32 * kQWarps), 0, stream, p, s, fault);
  }
  const uint32_t warps = (pairs + 3) / 4;
  return launch_after_predecessor(quantize_kernel<T, kMode, 4>, dim3((warps + kQWarps - 1) / kQWarps),
                                  dim3(32 * kQWarps), 0, stream, p, s, fault);
}

template <typename T>
cudaError_t launch_type(const qsfm_quantize_params& p, const QuantizeShape& s, int* fault, cudaStream_t stream) {
  if (p.gate != nullptr) return launch_mode<T, kGated>(p, s, fault, stream);
  if (p.rope_dim > 0) return launch_mode<T, kRotate>(p, s, fault, stream);
  return launch_mode<T, kPlain>(p, s, fault, stream);
}

}  // namespace

cudaError_t launch_quantize(const qsfm_quantize_params& p, int* fault, cudaStream_t stream) {
  QuantizeShape s;
  s.k = p.heads * p.dim;
  s.groups = uint32_t((s.k + kQGroup - 1) / kQGroup);
  s.total = uint32_t(p.rows) * s.groups;
  s.per_row.set(s.groups);
  s.per_head.set(p.heads > 1 ? uint32_t(p.dim / kQGroup) : 1);
  switch (p.in_type) {
    case QSFM_BF16: return launch_type<__nv_bfloat16>(p, s, fault, stream);
    case QSFM_F16: return launch_type<__half>(p, s, fault, stream);
    default: return launch_type<float>(p, s, fault, stream);
  }
}

}  // namespace qsfm
