// ibp_mx_matmul.hip -- product of microscaled tensors: y[m][n] = sum over k of
// A[m][k] B[n][k], A (activations) in e4m3 or e2m1, B (weights) in e2m1, sums in 32
// bits, one rounding to y's type.
//
// The matrix instruction takes 16 rows x 128 elements of each operand with a scale byte
// per row and 32 elements (v_mfma_scale_f32_16x16x128_f8f6f4); both operands lie along
// k as the packed format stores them, so a lane's operand is a 16-byte load.  Lane l
// holds row l % 16; with g = l / 16, an e2m1 lane holds block g of the four, an e4m3
// lane bytes [16 g, 16 g + 16) of blocks 0..1 and of blocks 2..3; the scale of block g
// is lane group g's.  Weights are the instruction's first operand, so a lane's four
// results are consecutive n of one m.
#include "ibp_device.h"
#include "ibp_num.h"

namespace ibp {
namespace {

using namespace dev;

typedef int v8i __attribute__((ext_vector_type(8)));

constexpr uint32_t kStep = 16;  // blocks per step of the direct kernel: 512 elements

template <bool A8> __device__ __forceinline__ v4f mfma_mx(v8i w, v8i x, v4f acc, int ws, int xs, int sel) {
  // format codes: 0 e4m3, 4 e2m1; sel: which byte of the scale words
  constexpr int fx = A8 ? 0 : 4;
  switch (sel) {
    case 0: return __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(w, x, acc, 4, fx, 0, ws, 0, xs);
    case 1: return __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(w, x, acc, 4, fx, 1, ws, 1, xs);
    case 2: return __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(w, x, acc, 4, fx, 2, ws, 2, xs);
    default: return __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(w, x, acc, 4, fx, 3, ws, 3, xs);
  }
}

// A 16-byte piece of a row, zero from byte `pitch` on.
__device__ __forceinline__ uint4 piece(const uint8_t *row, uint32_t at, uint32_t pitch) {
  return at < pitch ? *reinterpret_cast<const uint4 *>(row + at) : make_uint4(0u, 0u, 0u, 0u);
}

__device__ __forceinline__ v8i operand(uint4 lo, uint4 hi) {
  return v8i{(int)lo.x, (int)lo.y, (int)lo.z, (int)lo.w, (int)hi.x, (int)hi.y, (int)hi.z, (int)hi.w};
}

// Few rows of A: bound by the weights' bytes.  A workgroup computes 16 MI x 16 outputs,
// its wavefronts take the steps of k in turn and their sums are added in order through
// LDS.  A step covers 16 blocks, four matrix instructions of which instruction s takes
// blocks s, 4 + s, 8 + s, 12 + s (the sum over k may take its blocks in any order), so
// lane group g's weights are 64 consecutive bytes and its scales one dword.
template <bool A8, int MI, int DO> __global__ void mx_direct_kernel(MxMatmulArgs a) {
  using TO = typename Num<DO>::T;
  extern __shared__ float red[];
  const uint32_t lane = lane_id(), wave = uniform(threadIdx.x / kWave), waves = blockDim.x / kWave;
  const uint32_t r = lane & 15, g = lane >> 4;
  const uint64_t n0 = (uint64_t)blockIdx.x * 16, m0 = (uint64_t)blockIdx.y * (16 * MI);
  const uint32_t nblk = (uint32_t)mx_blocks(a.K), sp = (uint32_t)mx_scale_pitch(a.K);
  const uint32_t wp = (uint32_t)mx_code_pitch(a.K, false), xp = (uint32_t)mx_code_pitch(a.K, A8);
  // rows past the end repeat the last one; their results are not stored
  const uint64_t n = n0 + r < a.N ? n0 + r : a.N - 1;
  const uint8_t *wc = a.b_codes + n * wp, *wsc = a.b_scales + n * sp;
  const uint8_t *xc[MI], *xsc[MI];
#pragma unroll
  for (int i = 0; i < MI; ++i) {
    const uint64_t m = m0 + 16 * i + r < a.M ? m0 + 16 * i + r : a.M - 1;
    xc[i] = a.a_codes + m * xp;
    xsc[i] = a.a_scales + m * sp;
  }
  v4f acc[MI];
#pragma unroll
  for (int i = 0; i < MI; ++i) acc[i] = v4f{0, 0, 0, 0};
  for (uint32_t b0 = wave * kStep; b0 < nblk; b0 += waves * kStep) {
    const uint32_t sb = b0 + 4 * g;
    uint4 w[4];
#pragma unroll
    for (int s = 0; s < 4; ++s) w[s] = piece(wc, (sb + s) * 16, wp);
    const int ws = sb < sp ? *reinterpret_cast<const int *>(wsc + sb) : 0;
    int xs[MI];
#pragma unroll
    for (int i = 0; i < MI; ++i) xs[i] = sb < sp ? *reinterpret_cast<const int *>(xsc[i] + sb) : 0;
#pragma unroll
    for (int i = 0; i < MI; ++i) {
#pragma unroll
      for (int s = 0; s < 4; ++s) {
        uint4 lo, hi = make_uint4(0u, 0u, 0u, 0u);
        if constexpr (A8) {
          lo = piece(xc[i], (b0 + 4 * (g >> 1) + s) * 32 + 16 * (g & 1), xp);
          hi = piece(xc[i], (b0 + 4 * (2 + (g >> 1)) + s) * 32 + 16 * (g & 1), xp);
        } else {
          lo = piece(xc[i], (sb + s) * 16, xp);
        }
        acc[i] = mfma_mx<A8>(operand(w[s], make_uint4(0u, 0u, 0u, 0u)), operand(lo, hi), acc[i], ws, xs[i], s);
      }
    }
  }
  if (waves > 1) {
    if (wave) {
#pragma unroll
      for (int i = 0; i < MI; ++i)
        *reinterpret_cast<v4f *>(red + ((wave - 1) * MI + i) * 256 + lane * 4) = acc[i];
    }
    __syncthreads();
    if (wave) return;
    for (uint32_t w = 0; w + 1 < waves; ++w) {
#pragma unroll
      for (int i = 0; i < MI; ++i) acc[i] += *reinterpret_cast<const v4f *>(red + (w * MI + i) * 256 + lane * 4);
    }
  }
  TO *y = static_cast<TO *>(a.y);
#pragma unroll
  for (int i = 0; i < MI; ++i) {
    const uint64_t m = m0 + 16 * i + r;
    if (m < a.M) store4<TO>(y + m * a.N, n0 + 4 * g, a.N, acc[i]);
  }
}

template <bool A8, int MI> hipError_t go_direct(const MxMatmulArgs &a, hipStream_t s) {
  const uint64_t gx = (a.N + 15) / 16, gy = (a.M + 16 * MI - 1) / (16 * MI);
  const uint32_t steps = (uint32_t)((mx_blocks(a.K) + kStep - 1) / kStep);
  uint32_t waves = gx * gy < 512 ? 16 : 4;
  while (waves > 1 && waves > steps) waves /= 2;
  if (gx > 0xFFFFFF || gy > 0xFFFF) return hipErrorInvalidValue;
  return with_dtype(a.dtype, [&](auto d) {
    mx_direct_kernel<A8, MI, d.value>
        <<<dim3((uint32_t)gx, (uint32_t)gy), waves * kWave, (waves - 1) * MI * 1024, s>>>(a);
    return hipGetLastError();
  });
}

}  // namespace

uint64_t mx_matmul_workspace(uint64_t, uint64_t, uint32_t, bool) { return 0; }

hipError_t launch_mx_matmul(const MxMatmulArgs &a, hipStream_t s) {
  if (a.a_e4m3) return a.M <= 16 ? go_direct<true, 1>(a, s) : go_direct<true, 4>(a, s);
  return a.M <= 16 ? go_direct<false, 1>(a, s) : go_direct<false, 4>(a, s);
}

}  // namespace ibp
