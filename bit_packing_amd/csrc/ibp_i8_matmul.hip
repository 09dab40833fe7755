// ibp_i8_matmul.hip -- product of 8-bit integer rows: y[m][n] = sa[m] sb[n] sum over k of
// A[m][k] B[n][k], whole numbers summed in 32 bits, which hold 131071 products of any codes.
//
// The matrix instruction takes 16 rows x 64 codes of each operand (v_mfma_i32_16x16x64_i8);
// both operands lie along k, so a lane's operand is a 16-byte load: lane l holds codes [16 g,
// 16 g + 16) of row l % 16, g = l / 16.  Weights are the instruction's first operand, so a
// lane's four results are consecutive n of one m.  Sums of whole numbers do not depend on
// their order: k may be cut anywhere.
#include "ibp_device.h"
#include "ibp_num.h"
#include "ibp_tile.h"

namespace ibp {
namespace {

using namespace dev;

typedef int v4i __attribute__((ext_vector_type(4)));

__device__ __forceinline__ v4i mfma(v4i w, v4i x, v4i acc) { return __builtin_amdgcn_mfma_i32_16x16x64_i8(w, x, acc, 0, 0, 0); }

__device__ __forceinline__ v4i as_int(uint4 v) { return v4i{(int)v.x, (int)v.y, (int)v.z, (int)v.w}; }

// A sum times its scales, the smaller first: no product on the way is beyond the floats
// where the result is not.
__device__ __forceinline__ float scaled(int sum, float sa, float sb) {
  const bool a_less = fabsf(sa) < fabsf(sb);
  return (float)sum * (a_less ? sa : sb) * (a_less ? sb : sa);
}

// The scales of four columns from n on, zeros past the end.
__device__ __forceinline__ v4f scales4(const float *scales, uint64_t n, uint64_t N) { return load4(scales, n, N); }

__device__ __forceinline__ v4f scaled4(v4i sum, float sa, v4f sb) {
  return v4f{scaled(sum[0], sa, sb[0]), scaled(sum[1], sa, sb[1]), scaled(sum[2], sa, sb[2]), scaled(sum[3], sa, sb[3])};
}

// Few rows of A.  A workgroup computes 16 x 16 outputs, its wavefronts take steps of 256
// codes in turn.
constexpr uint32_t kStep = 256;
template <int DO> __global__ void i8_direct_kernel(I8MatmulArgs a) {
  using TO = typename Num<DO>::T;
  extern __shared__ int red[];
  const uint32_t lane = lane_id(), wave = uniform(threadIdx.x / kWave), waves = blockDim.x / kWave;
  const uint32_t r = lane & 15, g = lane >> 4, cp = (uint32_t)i8_pitch(a.K);
  const uint64_t n0 = (uint64_t)blockIdx.x * 16, m0 = (uint64_t)blockIdx.y * 16;
  // rows past the end repeat the last one; their results are not stored
  const uint64_t n = n0 + r < a.N ? n0 + r : a.N - 1, m = m0 + r < a.M ? m0 + r : a.M - 1;
  const uint8_t *wc = a.b_codes + n * cp, *xc = a.a_codes + m * cp;
  v4i acc{0, 0, 0, 0};
  for (uint32_t k = wave * kStep; k < cp; k += waves * kStep) {
    uint4 w[4], x[4];
#pragma unroll
    for (int s = 0; s < 4; ++s) w[s] = piece(wc, k + 64 * s + 16 * g, cp);
#pragma unroll
    for (int s = 0; s < 4; ++s) x[s] = piece(xc, k + 64 * s + 16 * g, cp);
#pragma unroll
    for (int s = 0; s < 4; ++s) acc = mfma(as_int(w[s]), as_int(x[s]), acc);
  }
  if (waves > 1) {
    if (wave) *reinterpret_cast<v4i *>(red + (wave - 1) * 256 + lane * 4) = acc;
    __syncthreads();
    if (wave) return;
    for (uint32_t k = 0; k + 1 < waves; ++k) acc += *reinterpret_cast<const v4i *>(red + k * 256 + lane * 4);
  }
  if (m0 + r < a.M)
    store4<TO>(static_cast<TO *>(a.y) + (m0 + r) * a.N, n0 + 4 * g, a.N,
               scaled4(acc, a.a_scales[m0 + r], scales4(a.b_scales, n0 + 4 * g, a.N)));
}

hipError_t go_direct(const I8MatmulArgs &a, hipStream_t s) {
  const uint64_t gx = (a.N + 15) / 16, gy = (a.M + 15) / 16;
  const uint32_t steps = (a.K + kStep - 1) / kStep;
  uint32_t waves = gx * gy <= 256 ? 16 : 4;
  while (waves > 1 && waves > steps) waves /= 2;
  return with_dtype(a.dtype, [&](auto d) {
    I8MatmulArgs part = a;
    for (uint64_t y0 = 0; y0 < gy; y0 += 65535) {
      const uint64_t n = gy - y0 < 65535 ? gy - y0 : 65535;
      i8_direct_kernel<d.value><<<dim3((uint32_t)gx, (uint32_t)n), waves * kWave, (waves - 1) * 1024, s>>>(part);
      part.M -= n * 16 < part.M ? n * 16 : part.M;
      part.a_codes += n * 16 * i8_pitch(a.K);
      part.a_scales += n * 16;
      part.y = static_cast<uint8_t *>(part.y) + n * 16 * a.N * sizeof(typename Num<d.value>::T);
    }
    return hipGetLastError();
  });
}

}  // namespace

uint64_t i8_matmul_workspace(uint64_t, uint64_t, uint32_t) { return 0; }

hipError_t launch_i8_matmul(const I8MatmulArgs &a, hipStream_t s) { return go_direct(a, s); }

}  // namespace ibp
