// ibp_num.h -- number formats of the language-model operators: float, half and
// bfloat16 tensors in vectors of eight elements, and the microscaled element types
// e4m3 and e2m1 with their power-of-two block scales.
#pragma once

#include <type_traits>

#include "ibp.h"
#include "ibp_ops.h"

namespace ibp {
namespace dev {

template <int D> struct Num;
template <> struct Num<IBP_F32> { using T = float; };
template <> struct Num<IBP_F16> { using T = _Float16; };
template <> struct Num<IBP_BF16> { using T = __bf16; };

// Eight elements at element alignment: rows of odd length start anywhere, and the
// global memory path takes unaligned wide accesses, so one form serves all rows.
template <typename T> struct VecOf { typedef T type __attribute__((ext_vector_type(8), aligned(sizeof(T)))); };
template <typename T> using Vec8 = typename VecOf<T>::type;

struct F8 { float v[8]; };

// x with its elements moved down by n (1..7), zeros moving in.
template <typename T> __device__ __forceinline__ Vec8<T> move_down(Vec8<T> x, uint32_t n) {
  constexpr int W = 2 * sizeof(T);  // dwords
  uint32_t d[W];
  __builtin_memcpy(d, &x, sizeof(d));
  if constexpr (sizeof(T) == 2) {
    if (n & 1) {
#pragma unroll
      for (int i = 0; i < W; ++i) d[i] = (d[i] >> 16) | (i + 1 < W ? d[i + 1] << 16 : 0u);
    }
    n >>= 1;
  }
#pragma unroll
  for (int k = 1; k < W; k *= 2) {
    const bool on = n & k;
#pragma unroll
    for (int i = 0; i < W; ++i) d[i] = on ? (i + k < W ? d[i + k] : 0u) : d[i];
  }
  __builtin_memcpy(&x, d, sizeof(d));
  return x;
}

// Elements [c, c + 8) of a row of `cols` elements are loaded by load8 as they lie in
// memory, and given zeros past the row's end by widen where they are used.  At the row's
// end load8 takes the row's last eight elements: one load for every lane and no branch,
// so that no load waits for another (element by element, or with the end's lanes in a
// branch of their own, each load of a wavefront at the end waited).  Rows of less than
// eight elements (WIDE false) are loaded one by one; a kernel asks once which it has
// (by_width), as even a uniform branch at each load makes the loads wait for each other.
template <bool WIDE, typename T> __device__ __forceinline__ Vec8<T> load8(const T *row, uint32_t c, uint32_t cols) {
  if constexpr (WIDE) {
    return *reinterpret_cast<const Vec8<T> *>(row + (c + 8 <= cols ? c : cols - 8));
  } else {
    Vec8<T> x = {};
#pragma unroll
    for (int i = 0; i < 7; ++i)
      if (i < (int)cols) x[i] = row[i];
    return x;
  }
}

template <bool WIDE, typename T> __device__ __forceinline__ Vec8<T> settle8(Vec8<T> x, uint32_t c, uint32_t cols) {
  if (c >= cols) return Vec8<T>{};
  if (WIDE && c + 8 > cols) return move_down<T>(x, c + 8 - cols);
  return x;
}

template <bool WIDE, typename T> __device__ __forceinline__ F8 widen(Vec8<T> x, uint32_t c, uint32_t cols) {
  x = settle8<WIDE, T>(x, c, cols);
  F8 r;
#pragma unroll
  for (int i = 0; i < 8; ++i) r.v[i] = (float)x[i];
  return r;
}

template <typename F> __device__ __forceinline__ void by_width(uint32_t cols, F &&f) {
  if (cols >= 8) f(std::true_type{});
  else f(std::false_type{});
}

// The same elements written, each rounded once to T (nearest, ties to even).
template <typename T> __device__ __forceinline__ void store8(T *row, uint32_t c, uint32_t cols, const F8 &r) {
  if (c + 8 <= cols) {
    Vec8<T> x;
#pragma unroll
    for (int i = 0; i < 8; ++i) x[i] = (T)r.v[i];
    *reinterpret_cast<Vec8<T> *>(row + c) = x;
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i)
      if (c + i < cols) row[c + i] = (T)r.v[i];
  }
}

typedef float v4f __attribute__((ext_vector_type(4)));

// Four consecutive elements at n of a row of N, each rounded once to TO.
template <typename TO>
__device__ __forceinline__ void store4(TO *row, uint64_t n, uint64_t N, v4f v) {
  if (n + 4 <= N) {
    typedef TO V __attribute__((ext_vector_type(4), aligned(sizeof(TO))));
    V o;
#pragma unroll
    for (int i = 0; i < 4; ++i) o[i] = (TO)v[i];
    *reinterpret_cast<V *>(row + n) = o;
  } else {
#pragma unroll
    for (int i = 0; i < 4; ++i)
      if (n + i < N) row[n + i] = (TO)v[i];
  }
}

__device__ __forceinline__ v4f load4(const float *row, uint64_t n, uint64_t N) {
  typedef float V __attribute__((ext_vector_type(4), aligned(4)));
  v4f v{0, 0, 0, 0};
  if (n + 4 <= N) {
    v = *reinterpret_cast<const V *>(row + n);
  } else {
#pragma unroll
    for (int i = 0; i < 4; ++i)
      if (n + i < N) v[i] = row[n + i];
  }
  return v;
}

// ------------------------------------------------------------------ microscaled blocks

constexpr int kMxMinExp = -117;  // smallest scale exponent: the smallest non-zero e4m3 value is then 2^-126, normal
constexpr uint32_t kMxNanScale = 255u;

// 2^e for -126 <= e <= 127.
__device__ __forceinline__ float pow2(int e) { return __builtin_bit_cast(float, (uint32_t)(e + 127) << 23); }

// Scale byte of a block whose largest magnitude has the float bits `amax` (sign
// clear): the smallest exponent s with |x| <= M 2^s, s + 127; M = 1.75 * 2^8 (e4m3)
// or 1.5 * 2^2 (e2m1), so s = exponent - 8 or - 2, one more when the fraction is
// above that of M.  255 when the block holds an infinity or a NaN.
template <bool E4M3> __device__ __forceinline__ uint32_t mx_scale(uint32_t amax) {
  if (amax >= 0x7F800000u) return kMxNanScale;
  const int e = (int)(amax >> 23) - (E4M3 ? 8 : 2) + ((amax & 0x7FFFFFu) > (E4M3 ? 0x600000u : 0x400000u) ? 1 : 0);
  const int lo = kMxMinExp + 127, hi = (E4M3 ? 119 : 125) + 127;
  return (uint32_t)(e < lo ? lo : (e > hi ? hi : e));
}

// Eight elements over the scale, rounded to codes (nearest, ties to even, saturating).
// e4m3: eight bytes; e2m1: eight nibbles in .x.  A block of scale 255 gets codes 0.
template <bool E4M3> __device__ __forceinline__ uint2 mx_encode(const F8 &x, uint32_t scale) {
  uint2 c = make_uint2(0u, 0u);
  if (scale == kMxNanScale) return c;
  const float inv = pow2(127 - (int)scale);  // exact: 127 - scale lies in [-125, 117]
  if constexpr (E4M3) {
    float y[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) y[i] = fminf(fmaxf(x.v[i] * inv, -448.0f), 448.0f);
    int a = __builtin_amdgcn_cvt_pk_fp8_f32(y[0], y[1], 0, false);
    a = __builtin_amdgcn_cvt_pk_fp8_f32(y[2], y[3], a, true);
    int b = __builtin_amdgcn_cvt_pk_fp8_f32(y[4], y[5], 0, false);
    b = __builtin_amdgcn_cvt_pk_fp8_f32(y[6], y[7], b, true);
    c.x = (uint32_t)a;
    c.y = (uint32_t)b;
  } else {
    // the conversion saturates at 6 by itself
    uint32_t a = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(0u, x.v[0] * inv, x.v[1] * inv, 1.0f, 0);
    a = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(a, x.v[2] * inv, x.v[3] * inv, 1.0f, 1);
    a = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(a, x.v[4] * inv, x.v[5] * inv, 1.0f, 2);
    a = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(a, x.v[6] * inv, x.v[7] * inv, 1.0f, 3);
    c.x = a;
  }
  return c;
}

// A block scale as a float factor; bytes below the smallest exponent the packer
// writes are taken as they are (2^-127 is a subnormal float).
__device__ __forceinline__ float mx_factor(uint32_t scale) {
  uint32_t bits = scale << 23;
  bits = scale == 0 ? 0x400000u : bits;
  bits = scale == kMxNanScale ? 0x7FC00000u : bits;
  return __builtin_bit_cast(float, bits);
}

// Values of eight codes (e4m3: eight bytes; e2m1: the nibbles of .x).
template <bool E4M3> __device__ __forceinline__ F8 mx_decode(uint2 c, uint32_t scale) {
  typedef float v2f __attribute__((ext_vector_type(2)));
  const float f = mx_factor(scale);
  F8 r;
  v2f p[4];
  if constexpr (E4M3) {
    p[0] = __builtin_amdgcn_cvt_pk_f32_fp8((int)c.x, false);
    p[1] = __builtin_amdgcn_cvt_pk_f32_fp8((int)c.x, true);
    p[2] = __builtin_amdgcn_cvt_pk_f32_fp8((int)c.y, false);
    p[3] = __builtin_amdgcn_cvt_pk_f32_fp8((int)c.y, true);
  } else {
    p[0] = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(c.x, 1.0f, 0);
    p[1] = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(c.x, 1.0f, 1);
    p[2] = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(c.x, 1.0f, 2);
    p[3] = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(c.x, 1.0f, 3);
  }
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    r.v[2 * i] = p[i][0] * f;
    r.v[2 * i + 1] = p[i][1] * f;
  }
  return r;
}

}  // namespace dev

// Calls f with the dtype as a compile-time constant.
template <typename F> hipError_t with_dtype(int dtype, F &&f) {
  switch (dtype) {
    case IBP_F32: return f(std::integral_constant<int, IBP_F32>{});
    case IBP_F16: return f(std::integral_constant<int, IBP_F16>{});
    case IBP_BF16: return f(std::integral_constant<int, IBP_BF16>{});
    default: return hipErrorInvalidValue;
  }
}

}  // namespace ibp
