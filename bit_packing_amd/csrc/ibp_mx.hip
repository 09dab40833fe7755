// ibp_mx.hip -- microscaled tensors: packing to e4m3 or e2m1 codes with one power-of-two
// scale per 32 elements, reading them back, and the gated activation silu(gate) * up
// that keeps its inputs as e4m3 checkpoints, with its backward pass from them.
//
// All four are one pass over the data, bound by HBM: 16384 x 8192 in bf16 is packed to e2m1
// and read back in 137 us (5.0 TB/s; a copy of 1 GiB reaches 5.2), packed to e4m3 in 73; the
// gated activation takes 185 us forward (5.8 TB/s) and 183 back (5.9).  A lane takes eight
// consecutive elements (16 bytes of a 16-bit type), so four lanes hold a block and share its
// largest magnitude by two lane exchanges, and 16 lanes hold the four blocks whose scale
// bytes make one dword.  A row is cut into strips of 8 times the smallest power of two of
// lanes, from 16 to the workgroup, that covers it; a workgroup step is one strip of R * 256
// / lanes rows, R of them per lane (one or four, where it packs or reads back), loaded before
// any is worked on.
#include "ibp_device.h"
#include "ibp_num.h"

namespace ibp {
namespace {

using namespace dev;

// Exchanges within a row of 16 lanes: lane ^ 1, lane ^ 2 (quad permutes), rotations by
// 4 and 8 lanes.
template <int CTRL> __device__ __forceinline__ uint32_t dpp(uint32_t v) {
  return (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, CTRL, 0xF, 0xF, false);
}
constexpr int kXor1 = 0xB1, kXor2 = 0x4E, kRor4 = 0x124, kRor8 = 0x128;

// Largest magnitude of the block that the lane's four-lane group holds, as float bits.
__device__ __forceinline__ uint32_t block_amax(const F8 &x) {
  uint32_t m = 0;
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const uint32_t b = __builtin_bit_cast(uint32_t, x.v[i]) & 0x7FFFFFFFu;  // ordered as integers, NaN on top
    m = b > m ? b : m;
  }
  uint32_t o = dpp<kXor1>(m);
  m = o > m ? o : m;
  o = dpp<kXor2>(m);
  return o > m ? o : m;
}

// One lane's eight elements at column c of a row into the row's codes and scales.
// All 16 lanes of the group call it; columns past the row's blocks write nothing, and
// their bytes of a scale dword are 0.
template <bool E4M3>
__device__ __forceinline__ void encode_lane(const F8 &x, uint8_t *codes, uint8_t *scales, uint32_t c, uint32_t nblk,
                                            bool row_ok) {
  const uint32_t scale = mx_scale<E4M3>(block_amax(x));
  const uint2 q = mx_encode<E4M3>(x, scale);
  const uint32_t blk = c / kMxBlock;
  uint32_t s = blk < nblk ? scale << (8 * (blk & 3)) : 0u;
  s |= dpp<kRor4>(s);
  s |= dpp<kRor8>(s);
  if (!row_ok || blk >= nblk) return;
  if constexpr (E4M3) *reinterpret_cast<uint2 *>(codes + c) = q;
  else *reinterpret_cast<uint32_t *>(codes + c / 2) = q.x;
  if ((c & 127) == 0) *reinterpret_cast<uint32_t *>(scales + blk) = s;
}

template <bool E4M3> __device__ __forceinline__ uint2 load_codes(const uint8_t *codes, uint32_t c) {
  if constexpr (E4M3) return *reinterpret_cast<const uint2 *>(codes + c);
  return make_uint2(*reinterpret_cast<const uint32_t *>(codes + c / 2), 0u);
}

// 1 / (1 + exp(-g)) of eight gates.  The 16-bit types take it from the hardware's exp2 and
// reciprocal (1 unit of the last place each), the argument's rounding made good by a factor: 6
// half units in all, far below the result's own rounding, for a third of the instructions
// (forward of 16384 x 8192 in bf16, four rows a lane, 204 us against 245 with the library's exp
// and a true quotient, which 32-bit results take).
//
// Where a wavefront has a gate below -80, whose exp(-g) may overflow and whose reciprocal is
// flushed to zero from -87.3 on, all its gates go by e = exp(-|g|), which fades out through the
// subnormal numbers: 1 / (1 + e), times e for negative g (7 half units).  For every gate that
// takes 213 us.
template <int D> __device__ __forceinline__ F8 sigmoid8(const F8 &g) {
  F8 s;
  if constexpr (D == IBP_F32) {
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const float e = expf(-fabsf(g.v[i]));
      s.v[i] = (g.v[i] < 0.0f ? e : 1.0f) / (1.0f + e);
    }
  } else {
    constexpr float kLog2e = 1.44269502162933349609375f, kLog2eRest = 1.925963033500011e-8f, kLn2 = 0.693147182f;
    float least = g.v[0];
#pragma unroll
    for (int i = 1; i < 8; ++i) least = fminf(least, g.v[i]);
    if (ballot(least < -80.0f) == 0) {
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const float x = fmaxf(-g.v[i], -200.0f);  // exp2 is 0 beyond
        const float t = x * kLog2e;
        const float rest = fmaf(x, kLog2eRest, fmaf(x, kLog2e, -t));
        const float e = __builtin_amdgcn_exp2f(t) * fmaf(rest, kLn2, 1.0f);
        s.v[i] = __builtin_amdgcn_rcpf(1.0f + e);
      }
    } else {
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const float x = -fminf(fabsf(g.v[i]), 200.0f);
        const float n = __builtin_rintf(x * kLog2e);
        const float f = fmaf(x, kLog2eRest, fmaf(x, kLog2e, -n));
        const float e = __builtin_ldexpf(__builtin_amdgcn_exp2f(f), (int)n), r = __builtin_amdgcn_rcpf(1.0f + e);
        s.v[i] = g.v[i] < 0.0f ? e * r : r;
      }
    }
  }
  return s;
}

struct Walk {
  uint32_t lanes;   // lanes a row, a power of two, 16..kBlock
  uint32_t strips;  // strips of lanes * 8 columns a row
  uint32_t units;   // strips of all groups of R * kBlock / lanes rows
};

// This lane's column and rows of one unit.
template <uint32_t R> struct Place {
  uint32_t c;
  uint64_t row[R];
  bool ok[R];
  __device__ __forceinline__ Place(const Walk &w, uint32_t unit, uint64_t rows) {
    const uint32_t group = unit / w.strips, strip = unit - group * w.strips, rows_blk = kBlock / w.lanes;
    c = (strip * w.lanes + (threadIdx.x & (w.lanes - 1))) * 8;
#pragma unroll
    for (uint32_t k = 0; k < R; ++k) {
      row[k] = ((uint64_t)group * R + k) * rows_blk + threadIdx.x / w.lanes;
      ok[k] = row[k] < rows;
      if (!ok[k]) row[k] = rows - 1;
    }
  }
};

template <int D, bool E4M3, uint32_t R> __global__ __launch_bounds__(kBlock) void mx_pack_kernel(MxArgs a, Walk w) {
  using T = typename Num<D>::T;
  const uint32_t nblk = (uint32_t)mx_blocks(a.cols);
  const uint64_t cp = mx_code_pitch(a.cols, E4M3), sp = mx_scale_pitch(a.cols);
  const T *in = static_cast<const T *>(a.in);
  by_width(a.cols, [&](auto wide) {
    for (uint32_t unit = blockIdx.x; unit < w.units; unit += gridDim.x) {
      const Place<R> p(w, unit, a.rows);
      Vec8<T> x[R];
#pragma unroll
      for (uint32_t k = 0; k < R; ++k) x[k] = load8<wide.value, T>(in + p.row[k] * a.cols, p.c, a.cols);
#pragma unroll
      for (uint32_t k = 0; k < R; ++k)
        encode_lane<E4M3>(widen<wide.value, T>(x[k], p.c, a.cols), a.codes + p.row[k] * cp, a.scales + p.row[k] * sp, p.c, nblk, p.ok[k]);
    }
  });
}

template <int D, bool E4M3, uint32_t R> __global__ __launch_bounds__(kBlock) void mx_unpack_kernel(MxArgs a, Walk w) {
  using T = typename Num<D>::T;
  const uint64_t cp = mx_code_pitch(a.cols, E4M3), sp = mx_scale_pitch(a.cols);
  T *out = static_cast<T *>(a.out);
  for (uint32_t unit = blockIdx.x; unit < w.units; unit += gridDim.x) {
    const Place<R> p(w, unit, a.rows);
    if (p.c >= a.cols) continue;
    uint2 q[R];
    uint32_t s[R];
#pragma unroll
    for (uint32_t k = 0; k < R; ++k) {
      q[k] = load_codes<E4M3>(a.codes + p.row[k] * cp, p.c);
      s[k] = a.scales[p.row[k] * sp + p.c / kMxBlock];
    }
#pragma unroll
    for (uint32_t k = 0; k < R; ++k)
      if (p.ok[k]) store8<T>(out + p.row[k] * a.cols, p.c, a.cols, mx_decode<E4M3>(q[k], s[k]));
  }
}

// h = g * sigmoid(g) * u in 32 bits from the inputs as they came; g and u packed.
template <int D> __global__ __launch_bounds__(kBlock) void mx_swiglu_kernel(MxArgs a, Walk w) {
  using T = typename Num<D>::T;
  const uint32_t nblk = (uint32_t)mx_blocks(a.cols);
  const uint64_t cp = mx_code_pitch(a.cols, true), sp = mx_scale_pitch(a.cols);
  const T *gate = static_cast<const T *>(a.in), *up = static_cast<const T *>(a.in2);
  T *h = static_cast<T *>(a.out);
  by_width(a.cols, [&](auto wide) {
    for (uint32_t unit = blockIdx.x; unit < w.units; unit += gridDim.x) {
      const Place<1> p(w, unit, a.rows);
      const uint64_t row = p.row[0];
      const Vec8<T> vg = load8<wide.value, T>(gate + row * a.cols, p.c, a.cols);
      const Vec8<T> vu = load8<wide.value, T>(up + row * a.cols, p.c, a.cols);
      const F8 g = widen<wide.value, T>(vg, p.c, a.cols), u = widen<wide.value, T>(vu, p.c, a.cols);
      encode_lane<true>(g, a.codes + row * cp, a.scales + row * sp, p.c, nblk, p.ok[0]);
      encode_lane<true>(u, a.codes2 + row * cp, a.scales2 + row * sp, p.c, nblk, p.ok[0]);
      F8 o = sigmoid8<D>(g);
#pragma unroll
      for (int i = 0; i < 8; ++i) o.v[i] = g.v[i] * o.v[i] * u.v[i];
      if (p.ok[0] && p.c < a.cols) store8<T>(h + row * a.cols, p.c, a.cols, o);
    }
  });
}

// With s = sigmoid(g): dgate = dh u s (1 + g (1 - s)), dup = dh g s, g and u read back
// from the checkpoints.
template <int D> __global__ __launch_bounds__(kBlock) void mx_swiglu_backward_kernel(MxArgs a, Walk w) {
  using T = typename Num<D>::T;
  const uint64_t cp = mx_code_pitch(a.cols, true), sp = mx_scale_pitch(a.cols);
  const T *dh = static_cast<const T *>(a.in2);
  T *dgate = static_cast<T *>(a.out), *dup = static_cast<T *>(a.out2);
  by_width(a.cols, [&](auto wide) {
    for (uint32_t unit = blockIdx.x; unit < w.units; unit += gridDim.x) {
      const Place<1> p(w, unit, a.rows);
      if (p.c >= a.cols || !p.ok[0]) continue;
      const uint64_t row = p.row[0];
      const uint2 qg = load_codes<true>(a.codes + row * cp, p.c), qu = load_codes<true>(a.codes2 + row * cp, p.c);
      const uint32_t sg = a.scales[row * sp + p.c / kMxBlock], su = a.scales2[row * sp + p.c / kMxBlock];
      const Vec8<T> vd = load8<wide.value, T>(dh + row * a.cols, p.c, a.cols);
      const F8 g = mx_decode<true>(qg, sg), u = mx_decode<true>(qu, su), d = widen<wide.value, T>(vd, p.c, a.cols);
      const F8 s = sigmoid8<D>(g);
      F8 og, ou;
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const float ds = d.v[i] * s.v[i];
        og.v[i] = ds * u.v[i] * (1.0f + g.v[i] * (1.0f - s.v[i]));
        ou.v[i] = ds * g.v[i];
      }
      store8<T>(dgate + row * a.cols, p.c, a.cols, og);
      store8<T>(dup + row * a.cols, p.c, a.cols, ou);
    }
  });
}

constexpr uint32_t kMaxGrid = 1u << 22;

bool walk_of(const MxArgs &a, uint32_t each, Walk *w) {
  const uint32_t need = (a.cols + 7) / 8;  // lanes that a row has work for
  w->lanes = 16;
  while (w->lanes < need && w->lanes < kBlock) w->lanes *= 2;
  w->strips = (need + w->lanes - 1) / w->lanes;
  const uint64_t rows = (uint64_t)(kBlock / w->lanes) * each, groups = (a.rows + rows - 1) / rows;
  const unsigned __int128 units = (unsigned __int128)groups * w->strips;
  if (units > 0xFFFFFFFFu - kMaxGrid) return false;
  w->units = (uint32_t)units;
  return true;
}

uint32_t grid_of(const Walk &w) { return w.units < kMaxGrid ? w.units : kMaxGrid; }

// Packing and reading back.  Rows per lane: four of a 16-bit type where that leaves the GPU
// full, so that small calls spread over the CUs; bf16 of 4096 columns, four rows against one:
// 512 units of four rows pack in 3.8 and 3.8 us, 256 in 3.4 and 3.0, 1024 in 4.9 and 5.4, 2048 in
// 7.8 and 9.2; 16384 x 8192 is packed to e2m1 in 61 and 65 and read back in 59 and 72.  One of
// fp32, whose rows are twice the registers (113 and 105, 150 and 119).
template <int D, typename F> hipError_t with_walk(const MxArgs &a, F &&f) {
  Walk w;
  if constexpr (D != IBP_F32) {
    if (!walk_of(a, 4, &w)) return hipErrorInvalidValue;
    if (w.units >= 1024) {
      f(std::integral_constant<uint32_t, 4>{}, w, grid_of(w));
      return hipGetLastError();
    }
  }
  if (!walk_of(a, 1, &w)) return hipErrorInvalidValue;
  f(std::integral_constant<uint32_t, 1>{}, w, grid_of(w));
  return hipGetLastError();
}

}  // namespace

hipError_t launch_mx_pack(const MxArgs &a, hipStream_t s) {
  return with_dtype(a.dtype, [&](auto d) {
    return with_walk<d.value>(a, [&](auto r, const Walk &w, uint32_t grid) {
      if (a.e4m3) mx_pack_kernel<d.value, true, r.value><<<grid, kBlock, 0, s>>>(a, w);
      else mx_pack_kernel<d.value, false, r.value><<<grid, kBlock, 0, s>>>(a, w);
    });
  });
}

hipError_t launch_mx_unpack(const MxArgs &a, hipStream_t s) {
  return with_dtype(a.dtype, [&](auto d) {
    return with_walk<d.value>(a, [&](auto r, const Walk &w, uint32_t grid) {
      if (a.e4m3) mx_unpack_kernel<d.value, true, r.value><<<grid, kBlock, 0, s>>>(a, w);
      else mx_unpack_kernel<d.value, false, r.value><<<grid, kBlock, 0, s>>>(a, w);
    });
  });
}

// The gated activation has more to do an element, and takes a row a lane (16384 x 8192 in
// bf16: 185 us forward against 191 with four rows, 183 backward against 194; 4000 x 4097 25
// against 28, 24 against 26; 8000 x 2048 22.0 against 24.4, 22.4 against 22.1).
hipError_t launch_mx_swiglu(const MxArgs &a, hipStream_t s) {
  Walk w;
  if (!walk_of(a, 1, &w)) return hipErrorInvalidValue;
  return with_dtype(a.dtype, [&](auto d) {
    mx_swiglu_kernel<d.value><<<grid_of(w), kBlock, 0, s>>>(a, w);
    return hipGetLastError();
  });
}

hipError_t launch_mx_swiglu_backward(const MxArgs &a, hipStream_t s) {
  Walk w;
  if (!walk_of(a, 1, &w)) return hipErrorInvalidValue;
  return with_dtype(a.dtype, [&](auto d) {
    mx_swiglu_backward_kernel<d.value><<<grid_of(w), kBlock, 0, s>>>(a, w);
    return hipGetLastError();
  });
}

}  // namespace ibp
