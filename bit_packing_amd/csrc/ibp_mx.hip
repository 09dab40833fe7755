// ibp_mx.hip -- microscaled tensors: packing to e4m3 or e2m1 codes with one power-of-two
// scale per 32 elements, reading them back, and the gated activation silu(gate) * up
// that keeps its inputs as e4m3 checkpoints, with its backward pass from them.
//
// All four are one pass over the data, bound by HBM.  A lane takes eight consecutive
// elements (16 bytes of a 16-bit type), so four lanes hold a block and share its
// largest magnitude by two lane exchanges, and 16 lanes hold the four blocks whose
// scale bytes make one dword.  A row is taken by the smallest power of two of lanes,
// from 16 to the workgroup, that covers it; kRowsEach rows per lane are loaded before
// any of them is worked on, so a wavefront keeps that many loads in flight.
#include "ibp_device.h"
#include "ibp_num.h"

namespace ibp {
namespace {

using namespace dev;

constexpr uint32_t kRowsEach = 4;

// Largest magnitude of the block that the lane's four-lane group holds, as float bits.
__device__ __forceinline__ uint32_t block_amax(const F8 &x) {
  uint32_t m = 0;
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const uint32_t b = __builtin_bit_cast(uint32_t, x.v[i]) & 0x7FFFFFFFu;  // ordered as integers, NaN on top
    m = b > m ? b : m;
  }
  uint32_t o = (uint32_t)__shfl_xor((int)m, 1, kWave);
  m = o > m ? o : m;
  o = (uint32_t)__shfl_xor((int)m, 2, kWave);
  return o > m ? o : m;
}

// One lane's eight elements at column c of a row into the row's codes and scales.
// All 16 lanes of the group call it; columns past the row's blocks write nothing but
// the padding bytes of the scale dword.
template <bool E4M3>
__device__ __forceinline__ void encode_lane(const F8 &x, uint8_t *codes, uint8_t *scales, uint32_t c, uint32_t nblk,
                                            bool row_ok) {
  const uint32_t scale = mx_scale<E4M3>(block_amax(x));
  const uint2 q = mx_encode<E4M3>(x, scale);
  const uint32_t blk = c / kMxBlock;
  // bytes of blocks past the row's end are 0
  uint32_t s = blk < nblk ? scale << (8 * (blk & 3)) : 0u;
  s |= (uint32_t)__shfl_xor((int)s, 4, kWave);
  s |= (uint32_t)__shfl_xor((int)s, 8, kWave);
  if (!row_ok) return;
  if (blk < nblk) {
    if constexpr (E4M3) *reinterpret_cast<uint2 *>(codes + c) = q;
    else *reinterpret_cast<uint32_t *>(codes + c / 2) = q.x;
  }
  if ((c & 127) == 0 && blk < nblk) *reinterpret_cast<uint32_t *>(scales + blk) = s;
}

template <bool E4M3> __device__ __forceinline__ uint2 load_codes(const uint8_t *codes, uint32_t c) {
  if constexpr (E4M3) return *reinterpret_cast<const uint2 *>(codes + c);
  return make_uint2(*reinterpret_cast<const uint32_t *>(codes + c / 2), 0u);
}

// Row and column walk shared by the kernels: `lanes` lanes a row, kRowsEach rows a lane.
struct Walk {
  uint32_t lanes;     // power of two, 16..kBlock
  uint32_t rows_blk;  // rows that a workgroup's lanes cover: kBlock / lanes
  uint64_t steps;     // workgroup steps of rows_blk * kRowsEach rows, walked by the grid
};

template <int D, bool E4M3>
__global__ __launch_bounds__(kBlock) void mx_pack_kernel(MxArgs a, Walk w) {
  using T = typename Num<D>::T;
  const uint32_t tx = threadIdx.x & (w.lanes - 1), ty = threadIdx.x / w.lanes;
  const uint32_t nblk = (uint32_t)mx_blocks(a.cols);
  const uint64_t cp = mx_code_pitch(a.cols, E4M3), sp = mx_scale_pitch(a.cols);
  const T *in = static_cast<const T *>(a.in);
  for (uint64_t step = blockIdx.x; step < w.steps; step += gridDim.x)
  for (uint32_t c0 = 0; c0 < nblk * kMxBlock; c0 += w.lanes * 8) {
    const uint64_t r0 = step * w.rows_blk * kRowsEach + ty;
    const uint32_t c = c0 + tx * 8;
    F8 x[kRowsEach];
#pragma unroll
    for (uint32_t k = 0; k < kRowsEach; ++k) {
      const uint64_t r = r0 + (uint64_t)k * w.rows_blk;
      x[k] = load8<T>(in + (r < a.rows ? r : 0) * a.cols, r < a.rows ? c : a.cols, a.cols);
    }
#pragma unroll
    for (uint32_t k = 0; k < kRowsEach; ++k) {
      const uint64_t r = r0 + (uint64_t)k * w.rows_blk;
      encode_lane<E4M3>(x[k], a.codes + r * cp, a.scales + r * sp, c, nblk, r < a.rows);
    }
  }
}

template <int D, bool E4M3>
__global__ __launch_bounds__(kBlock) void mx_unpack_kernel(MxArgs a, Walk w) {
  using T = typename Num<D>::T;
  const uint32_t tx = threadIdx.x & (w.lanes - 1), ty = threadIdx.x / w.lanes;
  const uint64_t cp = mx_code_pitch(a.cols, E4M3), sp = mx_scale_pitch(a.cols);
  T *out = static_cast<T *>(a.out);
  for (uint64_t step = blockIdx.x; step < w.steps; step += gridDim.x)
  for (uint32_t c0 = 0; c0 < a.cols; c0 += w.lanes * 8) {
    const uint64_t r0 = step * w.rows_blk * kRowsEach + ty;
    const uint32_t c = c0 + tx * 8;
    uint2 q[kRowsEach];
    uint32_t s[kRowsEach];
#pragma unroll
    for (uint32_t k = 0; k < kRowsEach; ++k) {
      const uint64_t r = r0 + (uint64_t)k * w.rows_blk;
      if (r < a.rows && c < a.cols) {
        q[k] = load_codes<E4M3>(a.codes + r * cp, c);
        s[k] = a.scales[r * sp + c / kMxBlock];
      }
    }
#pragma unroll
    for (uint32_t k = 0; k < kRowsEach; ++k) {
      const uint64_t r = r0 + (uint64_t)k * w.rows_blk;
      if (r < a.rows && c < a.cols) store8<T>(out + r * a.cols, c, a.cols, mx_decode<E4M3>(q[k], s[k]));
    }
  }
}

// h = g / (1 + exp(-g)) * u in 32 bits from the inputs as they came; g and u packed.
template <int D>
__global__ __launch_bounds__(kBlock) void mx_swiglu_kernel(MxArgs a, Walk w) {
  using T = typename Num<D>::T;
  const uint32_t tx = threadIdx.x & (w.lanes - 1), ty = threadIdx.x / w.lanes;
  const uint32_t nblk = (uint32_t)mx_blocks(a.cols);
  const uint64_t cp = mx_code_pitch(a.cols, true), sp = mx_scale_pitch(a.cols);
  const T *gate = static_cast<const T *>(a.in), *up = static_cast<const T *>(a.in2);
  T *h = static_cast<T *>(a.out);
  for (uint64_t step = blockIdx.x; step < w.steps; step += gridDim.x)
  for (uint32_t c0 = 0; c0 < nblk * kMxBlock; c0 += w.lanes * 8) {
    const uint64_t r0 = step * w.rows_blk * kRowsEach + ty;
    const uint32_t c = c0 + tx * 8;
    F8 g[kRowsEach], u[kRowsEach];
#pragma unroll
    for (uint32_t k = 0; k < kRowsEach; ++k) {
      const uint64_t r = r0 + (uint64_t)k * w.rows_blk;
      const uint64_t at = (r < a.rows ? r : 0) * a.cols;
      g[k] = load8<T>(gate + at, r < a.rows ? c : a.cols, a.cols);
      u[k] = load8<T>(up + at, r < a.rows ? c : a.cols, a.cols);
    }
#pragma unroll
    for (uint32_t k = 0; k < kRowsEach; ++k) {
      const uint64_t r = r0 + (uint64_t)k * w.rows_blk;
      encode_lane<true>(g[k], a.codes + r * cp, a.scales + r * sp, c, nblk, r < a.rows);
      encode_lane<true>(u[k], a.codes2 + r * cp, a.scales2 + r * sp, c, nblk, r < a.rows);
      F8 o;
#pragma unroll
      for (int i = 0; i < 8; ++i) o.v[i] = g[k].v[i] / (1.0f + expf(-g[k].v[i])) * u[k].v[i];
      if (r < a.rows && c < a.cols) store8<T>(h + r * a.cols, c, a.cols, o);
    }
  }
}

// With s = 1 / (1 + exp(-g)): dgate = dh u s (1 + g (1 - s)), dup = dh g s, g and u read
// back from the checkpoints.
template <int D>
__global__ __launch_bounds__(kBlock) void mx_swiglu_backward_kernel(MxArgs a, Walk w) {
  using T = typename Num<D>::T;
  const uint32_t tx = threadIdx.x & (w.lanes - 1), ty = threadIdx.x / w.lanes;
  const uint64_t cp = mx_code_pitch(a.cols, true), sp = mx_scale_pitch(a.cols);
  const T *dh = static_cast<const T *>(a.in2);
  T *dgate = static_cast<T *>(a.out), *dup = static_cast<T *>(a.out2);
  for (uint64_t step = blockIdx.x; step < w.steps; step += gridDim.x)
  for (uint32_t c0 = 0; c0 < a.cols; c0 += w.lanes * 8) {
    const uint64_t r0 = step * w.rows_blk * kRowsEach + ty;
    const uint32_t c = c0 + tx * 8;
    uint2 qg[kRowsEach], qu[kRowsEach];
    uint32_t sg[kRowsEach], su[kRowsEach];
    F8 d[kRowsEach];
#pragma unroll
    for (uint32_t k = 0; k < kRowsEach; ++k) {
      const uint64_t r = r0 + (uint64_t)k * w.rows_blk;
      if (r < a.rows && c < a.cols) {
        qg[k] = load_codes<true>(a.codes + r * cp, c);
        qu[k] = load_codes<true>(a.codes2 + r * cp, c);
        sg[k] = a.scales[r * sp + c / kMxBlock];
        su[k] = a.scales2[r * sp + c / kMxBlock];
        d[k] = load8<T>(dh + r * a.cols, c, a.cols);
      }
    }
#pragma unroll
    for (uint32_t k = 0; k < kRowsEach; ++k) {
      const uint64_t r = r0 + (uint64_t)k * w.rows_blk;
      if (r < a.rows && c < a.cols) {
        const F8 g = mx_decode<true>(qg[k], sg[k]), u = mx_decode<true>(qu[k], su[k]);
        F8 og, ou;
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          const float s = 1.0f / (1.0f + expf(-g.v[i]));
          og.v[i] = d[k].v[i] * u.v[i] * s * (1.0f + g.v[i] * (1.0f - s));
          ou.v[i] = d[k].v[i] * g.v[i] * s;
        }
        store8<T>(dgate + r * a.cols, c, a.cols, og);
        store8<T>(dup + r * a.cols, c, a.cols, ou);
      }
    }
  }
}

uint32_t walk_of(const MxArgs &a, Walk *w) {
  const uint32_t need = (a.cols + 7) / 8;  // lanes that a row has work for
  w->lanes = 16;
  while (w->lanes < need && w->lanes < kBlock) w->lanes *= 2;
  w->rows_blk = kBlock / w->lanes;
  const uint64_t each = (uint64_t)w->rows_blk * kRowsEach;
  w->steps = (a.rows + each - 1) / each;
  return (uint32_t)(w->steps < (1u << 22) ? w->steps : (1u << 22));
}

}  // namespace

hipError_t launch_mx_pack(const MxArgs &a, hipStream_t s) {
  Walk w;
  const uint32_t blocks = walk_of(a, &w);
  return with_dtype(a.dtype, [&](auto d) {
    if (a.e4m3) mx_pack_kernel<d.value, true><<<blocks, kBlock, 0, s>>>(a, w);
    else mx_pack_kernel<d.value, false><<<blocks, kBlock, 0, s>>>(a, w);
    return hipGetLastError();
  });
}

hipError_t launch_mx_unpack(const MxArgs &a, hipStream_t s) {
  Walk w;
  const uint32_t blocks = walk_of(a, &w);
  return with_dtype(a.dtype, [&](auto d) {
    if (a.e4m3) mx_unpack_kernel<d.value, true><<<blocks, kBlock, 0, s>>>(a, w);
    else mx_unpack_kernel<d.value, false><<<blocks, kBlock, 0, s>>>(a, w);
    return hipGetLastError();
  });
}

hipError_t launch_mx_swiglu(const MxArgs &a, hipStream_t s) {
  Walk w;
  const uint32_t blocks = walk_of(a, &w);
  return with_dtype(a.dtype, [&](auto d) {
    mx_swiglu_kernel<d.value><<<blocks, kBlock, 0, s>>>(a, w);
    return hipGetLastError();
  });
}

hipError_t launch_mx_swiglu_backward(const MxArgs &a, hipStream_t s) {
  Walk w;
  const uint32_t blocks = walk_of(a, &w);
  return with_dtype(a.dtype, [&](auto d) {
    mx_swiglu_backward_kernel<d.value><<<blocks, kBlock, 0, s>>>(a, w);
    return hipGetLastError();
  });
}

}  // namespace ibp
