// ibp_i8.hip -- 8-bit integer rows with a scale each: codes 127 x / m, m the row's largest
// magnitude, rounded to the nearest whole number, and reading them back.
//
// Both are one pass over the data, bound by HBM: 16384 x 8192 in bf16 is packed in 81 us (5.0
// TB/s; a copy of 1 GiB reaches 5.0) and read back in 75.  A row belongs to a power of two of
// lanes, 16 to 256 or 1024, each with eight elements of every strip of 8 * lanes columns; a lane
// keeps what it has of a few strips in registers between the search for m and the rounding,
// longer rows are read twice.
#include "ibp_device.h"
#include "ibp_num.h"

namespace ibp {
namespace {

using namespace dev;

// The codes of eight elements.  127 x / m in 32 bits is off by less than 2^-22.9 of itself and
// a whole number and a half may come out as something next to it, so the quotient itself would
// not be rounded.  But a quotient of numbers of 11 or fewer bits that is no such border lies at
// least 1 / (254 * 2^11) > 2^-19 of itself from one, and the borders have at most 8 bits: cut
// to 21 bits, by which it moves at most 2^-21, it is on the border or on its side of it.  For
// 32-bit elements the same in 64 bits: at least 1 / (254 * 2^24) > 2^-32 apart, held on a grid
// of 2^-36.  Nearest, ties to even, comes from the addition of 1.5 * 2^23 (2^52), whose sum has
// the whole number in its low bits.
template <int D> struct Codes;
template <> struct Codes<IBP_F32> {
  double by;  // 127 / m
  __device__ __forceinline__ explicit Codes(float m) : by(m > 0.0f ? 127.0 / (double)m : 0.0) {}
  __device__ __forceinline__ uint32_t one(float x) const {
    constexpr double kGrid = 1.5 * 65536.0, kWhole = 1.5 * 4503599627370496.0;
    const double t = __dadd_rn(__dadd_rn(__dmul_rn((double)x, by), kGrid), -kGrid);
    return (uint32_t)__builtin_bit_cast(uint64_t, __dadd_rn(t, kWhole));
  }
};
struct Codes16 {
  float lift, by;  // 127 / m as lift * by: for the smallest m no float holds it
  __device__ __forceinline__ explicit Codes16(float m) {
    lift = m < 0x1p-100f ? 0x1p100f : 1.0f;
    by = m > 0.0f ? 127.0f / (m * lift) : 0.0f;
  }
  __device__ __forceinline__ uint32_t one(float x) const {
    const float t = __fmul_rn(__fmul_rn(x, lift), by);
    const uint32_t cut = (__builtin_bit_cast(uint32_t, t) + 4u) & ~7u;
    return __builtin_bit_cast(uint32_t, __fadd_rn(__builtin_bit_cast(float, cut), 12582912.0f));
  }
};
template <> struct Codes<IBP_F16> : Codes16 { using Codes16::Codes16; };
template <> struct Codes<IBP_BF16> : Codes16 { using Codes16::Codes16; };

template <int D> __device__ __forceinline__ uint2 codes8(const F8 &x, const Codes<D> &c) {
  uint32_t q[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) q[i] = c.one(x.v[i]);
  auto four = [](const uint32_t *q) {  // their low bytes
    const uint32_t a = __builtin_amdgcn_perm(q[1], q[0], 0x0C0C0400u), b = __builtin_amdgcn_perm(q[3], q[2], 0x0C0C0400u);
    return a | b << 16;
  };
  return make_uint2(four(q), four(q + 4));
}

// The largest float that a code of 127 times it leaves finite; the largest float over 127 is
// rounded to the one above.
constexpr float kMaxScale = 0x1.020406p+121f;

__device__ __forceinline__ uint32_t larger(uint32_t a, uint32_t b) { return a > b ? a : b; }

// R strips a row, kept in registers; 0: any number, read twice.
template <int D, uint32_t THREADS, uint32_t R>
__global__ __launch_bounds__(THREADS) void i8_pack_kernel(I8Args a, uint32_t lanes, uint32_t strips) {
  using T = typename Num<D>::T;
  __shared__ uint32_t tops[2][THREADS / kWave];
  const uint32_t tx = threadIdx.x & (lanes - 1), ty = threadIdx.x / lanes, rows_blk = THREADS / lanes;
  const uint32_t cp = (uint32_t)i8_pitch(a.cols), wave = uniform(threadIdx.x / kWave);
  const T *in = static_cast<const T *>(a.in);
  uint32_t odd = 0;
  by_width(a.cols, [&](auto wide) {
    for (uint64_t r0 = (uint64_t)blockIdx.x * rows_blk; r0 < a.rows; r0 += (uint64_t)gridDim.x * rows_blk) {
      const bool ok = r0 + ty < a.rows;
      const uint64_t row = ok ? r0 + ty : a.rows - 1;
      const T *from = in + row * a.cols;
      constexpr uint32_t kKept = R ? R : 1;
      Vec8<T> x[kKept];
      uint32_t m = 0;
      auto top = [&](const Vec8<T> &v, uint32_t c) {
        const F8 f = widen<wide.value, T>(v, c, a.cols);
#pragma unroll
        for (int i = 0; i < 8; ++i) m = larger(m, __builtin_bit_cast(uint32_t, f.v[i]) & 0x7FFFFFFFu);  // NaN on top
      };
      if constexpr (R > 0) {
#pragma unroll
        for (uint32_t k = 0; k < R; ++k) x[k] = load8<wide.value, T>(from, (k * lanes + tx) * 8, a.cols);
#pragma unroll
        for (uint32_t k = 0; k < R; ++k) top(x[k], (k * lanes + tx) * 8);
      } else {
        for (uint32_t k = 0; k < strips; ++k) {
          const uint32_t c = (k * lanes + tx) * 8;
          top(load8<wide.value, T>(from, c, a.cols), c);
        }
      }
      for (uint32_t o = 1; o < lanes && o < kWave; o *= 2) m = larger(m, (uint32_t)__shfl_xor((int)m, (int)o, kWave));
      if (lanes > kWave) {  // for the whole workgroup: its wavefronts share rows
        if (lane_id() == 0) tops[odd][wave] = m;
        __syncthreads();
        const uint32_t w0 = ty * (lanes / kWave);
        for (uint32_t w = 0; w < lanes / kWave; ++w) m = larger(m, tops[odd][w0 + w]);
        odd ^= 1;  // the next row's go elsewhere, so one barrier a row is enough
      }
      const bool fine = m < 0x7F800000u;
      const float amax = fine ? __builtin_bit_cast(float, m) : 0.0f;
      const Codes<D> by(amax);
      auto put = [&](const Vec8<T> &v, uint32_t c) {
        if (!ok || c >= cp) return;
        const uint2 q = codes8<D>(widen<wide.value, T>(v, c, a.cols), by);
        *reinterpret_cast<uint2 *>(a.codes + row * cp + c) = fine ? q : make_uint2(0u, 0u);
      };
      if constexpr (R > 0) {
#pragma unroll
        for (uint32_t k = 0; k < R; ++k) put(x[k], (k * lanes + tx) * 8);
      } else {
        for (uint32_t k = 0; k < strips; ++k) {
          const uint32_t c = (k * lanes + tx) * 8;
          put(load8<wide.value, T>(from, c, a.cols), c);
        }
      }
      if (ok && tx == 0) a.scales[row] = fine ? fminf(amax / 127.0f, kMaxScale) : __builtin_bit_cast(float, 0x7FC00000u);
    }
  });
}

// A code times its row's scale, rounded to 32 bits and then to T, as a float product and a
// conversion are.
template <int D> __global__ __launch_bounds__(kBlock) void i8_unpack_kernel(I8Args a, uint32_t lanes, uint32_t strips) {
  using T = typename Num<D>::T;
  const uint32_t tx = threadIdx.x & (lanes - 1), ty = threadIdx.x / lanes, rows_blk = kBlock / lanes;
  const uint32_t cp = (uint32_t)i8_pitch(a.cols);
  T *out = static_cast<T *>(a.out);
  const uint64_t units = (a.rows + rows_blk - 1) / rows_blk * strips;
  for (uint64_t unit = blockIdx.x; unit < units; unit += gridDim.x) {
    const uint64_t group = unit / strips, row = group * rows_blk + ty;
    const uint32_t c = ((uint32_t)(unit - group * strips) * lanes + tx) * 8;
    if (row >= a.rows || c >= a.cols) continue;
    const uint2 q = *reinterpret_cast<const uint2 *>(a.codes + row * cp + c);
    const float s = a.scales[row];
    auto four = [s](uint32_t q) {
      v4f v;
#pragma unroll
      for (int i = 0; i < 4; ++i) v[i] = (float)(int8_t)(q >> (8 * i)) * s;
      return as_floats(v);
    };
    const v4f lo = four(q.x), hi = four(q.y);
    const F8 v{{lo[0], lo[1], lo[2], lo[3], hi[0], hi[1], hi[2], hi[3]}};
    store8<T>(out + row * a.cols, c, a.cols, v);
  }
}

// Lanes that take a row, up to `most`, and the strips that cover it (its fill to 16 bytes with it).
void row_lanes(uint32_t cols, uint32_t most, uint32_t *lanes, uint32_t *strips) {
  const uint32_t need = (uint32_t)(i8_pitch(cols) / 8);
  *lanes = 16;
  while (*lanes < need && *lanes < most) *lanes *= 2;
  *strips = (need + *lanes - 1) / *lanes;
}

uint32_t grid_of(uint64_t units) { return (uint32_t)(units < (1u << 20) ? units : 1u << 20); }

}  // namespace

hipError_t launch_i8_pack(const I8Args &a, hipStream_t s) {
  return with_dtype(a.dtype, [&](auto d) {
    // Rows of more strips than registers hold well take a workgroup of sixteen wavefronts (4096 x
    // 16384: single precision 98 us with 256 lanes and eight strips, 75 with 1024 and two; bf16 42
    // and 60; 8192 x 8192 in single precision 67 with 256 and four, 99 with 1024 and one; 2048 x
    // 32768 in bf16 43 with 1024 and four).  A few rows would be quicker with them sooner (64 x
    // 16384 in bf16 5.3 and 4.7).
    constexpr bool kSingle = d.value == IBP_F32;
    constexpr uint32_t kLong = 1024, kStrips = kSingle ? 4 : 8, kLongStrips = kSingle ? 2 : 4;
    uint32_t lanes, strips, threads = kBlock;
    row_lanes(a.cols, kBlock, &lanes, &strips);
    if (strips > kStrips) row_lanes(a.cols, threads = kLong, &lanes, &strips);
    const uint64_t rows_blk = threads / lanes;
    auto launch = [&](auto kernel) { kernel<<<grid_of((a.rows + rows_blk - 1) / rows_blk), threads, 0, s>>>(a, lanes, strips); };
    if (threads == kLong) strips <= kLongStrips ? launch(i8_pack_kernel<d.value, kLong, kLongStrips>) : launch(i8_pack_kernel<d.value, kLong, 0>);
    else if (strips <= 1) launch(i8_pack_kernel<d.value, kBlock, 1>);
    else if (strips <= 2) launch(i8_pack_kernel<d.value, kBlock, 2>);
    else if (strips <= 4) launch(i8_pack_kernel<d.value, kBlock, 4>);
    else launch(i8_pack_kernel<d.value, kBlock, kStrips>);
    return hipGetLastError();
  });
}

hipError_t launch_i8_unpack(const I8Args &a, hipStream_t s) {
  uint32_t lanes, strips;
  row_lanes(a.cols, kBlock, &lanes, &strips);
  const uint64_t rows_blk = kBlock / lanes;
  const uint32_t grid = grid_of((a.rows + rows_blk - 1) / rows_blk * strips);
  return with_dtype(a.dtype, [&](auto d) {
    i8_unpack_kernel<d.value><<<grid, kBlock, 0, s>>>(a, lanes, strips);
    return hipGetLastError();
  });
}

}  // namespace ibp
