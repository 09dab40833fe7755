// ibp_mx_wgrad.hip -- weight gradient of a linear layer from the 8-bit checkpoint of its
// input: dW[o][i] = sum over tokens t of dY[t][o] X[t][i], dY in BF16, X packed as e4m3.
//
// An e4m3 value times its power-of-two scale (at least 2^-117) is a BF16 number, so X
// is decoded exactly to BF16 and the product runs on the BF16 matrix instruction with
// 32-bit sums.  Both operands lie with t as the slow dimension, while the instruction
// wants consecutive t in a lane: tiles are staged in LDS as they lie and read through
// the transposing LDS read, which hands each of 16 lanes one column of a 4 x 16 block.
#include "ibp_device.h"
#include "ibp_num.h"

namespace ibp {
namespace {

using namespace dev;

typedef short v4s __attribute__((ext_vector_type(4)));
typedef __bf16 v8b __attribute__((ext_vector_type(8)));

constexpr uint32_t kT = 32;  // tokens per stage

// LDS byte of the 16-byte piece `c16` of row t of a tile of `W` columns.  The 32-byte
// pieces of a row are permuted by the low bits of t: a transposing read takes 32 bytes
// of each of eight rows at a time, which then fall into all 64 banks.
template <uint32_t W> __device__ __forceinline__ uint32_t tile_at(uint32_t t, uint32_t c16) {
  return t * (W * 2) + ((((c16 >> 1) ^ (t & 7)) << 5) | ((c16 & 1) << 4));
}

// Eight BF16 of column block `col` (16 columns) in the order of the matrix
// instruction's k: lane group g takes rows 4 g .. 4 g + 3 and 16 + 4 g .. 16 + 4 g + 3.
template <uint32_t W> __device__ __forceinline__ v8b fragment(const uint8_t *tile, uint32_t col, uint32_t lane) {
  const uint32_t t = (lane >> 4) * 4 + ((lane & 15) >> 2), sub = (lane & 3) * 8;
  using L = __attribute__((address_space(3))) v4s;
  v4s lo = __builtin_amdgcn_ds_read_tr16_b64_v4i16((L *)(tile + t * (W * 2) + ((col ^ (t & 7)) << 5) + sub));
  v4s hi = __builtin_amdgcn_ds_read_tr16_b64_v4i16((L *)(tile + (t + 16) * (W * 2) + ((col ^ (t & 7)) << 5) + sub));
  typedef short v8s __attribute__((ext_vector_type(8)));
  const v8s v = __builtin_shufflevector(lo, hi, 0, 1, 2, 3, 4, 5, 6, 7);
  return __builtin_bit_cast(v8b, v);
}

// A workgroup of 2 x 2 wavefronts computes 32 F x 32 F of dW (o x i) over one range of
// tokens; with more than one range the sums go to the workspace in 32 bits.
template <int F, int DO, bool SPLIT>
__global__ __launch_bounds__(kBlock) void wgrad_kernel(MxWgradArgs a, uint64_t t_each) {
  using TO = typename Num<DO>::T;
  constexpr uint32_t W = 32 * F;                      // tile width, both ways
  constexpr uint32_t kPieces = kT * W / 8 / kBlock;   // eight-element pieces per thread and operand
  __shared__ __align__(16) uint8_t ty[kT * W * 2];
  __shared__ __align__(16) uint8_t tx[kT * W * 2];
  const uint32_t lane = lane_id(), wave = uniform(threadIdx.x / kWave);
  const uint32_t o0 = blockIdx.y * W, i0 = blockIdx.x * W;
  const uint32_t wo = (wave >> 1) * (W / 2), wi = (wave & 1) * (W / 2);
  const uint64_t t0 = blockIdx.z * t_each;
  const uint64_t t1 = t0 + t_each < a.T ? t0 + t_each : a.T;
  const uint64_t cp = mx_code_pitch(a.K, true), sp = mx_scale_pitch(a.K);
  const __bf16 *dy = static_cast<const __bf16 *>(a.dy);
  v4f acc[F][F];  // [i block][o block]
#pragma unroll
  for (int x = 0; x < F; ++x)
#pragma unroll
    for (int y = 0; y < F; ++y) acc[x][y] = v4f{0, 0, 0, 0};
  for (uint64_t tb = t0; tb < t1; tb += kT) {
    v8b vy[kPieces];
    uint2 qx[kPieces];
    uint32_t sx[kPieces];
#pragma unroll
    for (uint32_t p = 0; p < kPieces; ++p) {
      const uint32_t e = p * kBlock + threadIdx.x, t = e / (W / 8), c = e % (W / 8) * 8;
      const uint64_t tt = tb + t;
      vy[p] = v8b{};
      qx[p] = make_uint2(0u, 0u);
      sx[p] = 127u;
      if (tt < t1) {
        if (o0 + c + 8 <= a.N) {
          vy[p] = *reinterpret_cast<const Vec8<__bf16> *>(dy + tt * a.N + o0 + c);
        } else {
#pragma unroll
          for (int i = 0; i < 8; ++i)
            if (o0 + c + i < a.N) vy[p][i] = dy[tt * a.N + o0 + c + i];
        }
        if (i0 + c < cp) {
          qx[p] = *reinterpret_cast<const uint2 *>(a.x_codes + tt * cp + i0 + c);
          sx[p] = a.x_scales[tt * sp + (i0 + c) / kMxBlock];
        }
      }
    }
    __syncthreads();
#pragma unroll
    for (uint32_t p = 0; p < kPieces; ++p) {
      const uint32_t e = p * kBlock + threadIdx.x, t = e / (W / 8), c16 = e % (W / 8);
      *reinterpret_cast<v8b *>(ty + tile_at<W>(t, c16)) = vy[p];
      const F8 f = mx_decode<true>(qx[p], sx[p]);
      v8b vx;
#pragma unroll
      for (int i = 0; i < 8; ++i) vx[i] = (__bf16)f.v[i];
      *reinterpret_cast<v8b *>(tx + tile_at<W>(t, c16)) = vx;
    }
    __syncthreads();
    v8b fy[F];
#pragma unroll
    for (int y = 0; y < F; ++y) fy[y] = fragment<W>(ty, wo / 16 + y, lane);
#pragma unroll
    for (int x = 0; x < F; ++x) {
      const v8b fx = fragment<W>(tx, wi / 16 + x, lane);
#pragma unroll
      for (int y = 0; y < F; ++y) acc[x][y] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(fx, fy[y], acc[x][y], 0, 0, 0);
    }
  }
  // a lane has four consecutive i of one o
#pragma unroll
  for (int y = 0; y < F; ++y) {
    const uint32_t o = o0 + wo + 16 * y + (lane & 15);
    if (o >= a.N) continue;
#pragma unroll
    for (int x = 0; x < F; ++x) {
      const uint32_t i = i0 + wi + 16 * x + 4 * (lane >> 4);
      if constexpr (SPLIT) store4<float>(a.ws + ((uint64_t)blockIdx.z * a.N + o) * a.K, i, a.K, acc[x][y]);
      else store4<TO>(static_cast<TO *>(a.dw) + (uint64_t)o * a.K, i, a.K, acc[x][y]);
    }
  }
}

// Adds the ranges' sums in order.
template <int DO> __global__ __launch_bounds__(kBlock) void wgrad_join_kernel(MxWgradArgs a, uint32_t splits) {
  using TO = typename Num<DO>::T;
  const uint64_t n = (uint64_t)a.N * a.K;
  for (uint64_t e = ((uint64_t)blockIdx.x * kBlock + threadIdx.x) * 4; e < n; e += (uint64_t)gridDim.x * kBlock * 4) {
    v4f s{0, 0, 0, 0};
    for (uint32_t k = 0; k < splits; ++k) s += load4(a.ws + k * n, e, n);
    store4<TO>(static_cast<TO *>(a.dw), e, n, s);
  }
}

struct Plan {
  int F;            // 16-wide blocks a wavefront takes each way
  uint32_t splits;  // ranges of tokens
  uint64_t t_each;
};

Plan plan_of(uint64_t T, uint32_t N, uint32_t K) {
  Plan p;
  p.F = 4;
  const uint64_t W = 32 * p.F, tiles = ((N + W - 1) / W) * ((K + W - 1) / W);
  // enough workgroups for every CU twice, at least 256 tokens each
  const uint64_t want = tiles ? 512 / tiles : 1, most = (T + 255) / 256;
  uint64_t sp = want < most ? want : most;
  if (sp < 1) sp = 1;
  p.t_each = ((T + sp - 1) / sp + kT - 1) / kT * kT;
  if (p.t_each == 0) p.t_each = kT;
  p.splits = (uint32_t)((T + p.t_each - 1) / p.t_each);
  if (p.splits < 1) p.splits = 1;
  return p;
}

}  // namespace

uint64_t mx_wgrad_workspace(uint64_t T, uint32_t N, uint32_t K) {
  const Plan p = plan_of(T, N, K);
  return p.splits > 1 ? (uint64_t)p.splits * N * K * 4 : 0;
}

hipError_t launch_mx_wgrad(const MxWgradArgs &a, hipStream_t s) {
  const Plan p = plan_of(a.T, a.N, a.K);
  const uint32_t W = 32 * p.F;
  const dim3 grid((a.K + W - 1) / W, (a.N + W - 1) / W, p.splits);
  return with_dtype(a.dtype, [&](auto d) {
    if (p.splits == 1) {
      wgrad_kernel<4, d.value, false><<<grid, kBlock, 0, s>>>(a, p.t_each);
      return hipGetLastError();
    }
    wgrad_kernel<4, d.value, true><<<grid, kBlock, 0, s>>>(a, p.t_each);
    hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
    const uint64_t n = ((uint64_t)a.N * a.K + kBlock * 4 - 1) / (kBlock * 4);
    wgrad_join_kernel<d.value><<<(uint32_t)(n < 4096 ? n : 4096), kBlock, 0, s>>>(a, p.splits);
    return hipGetLastError();
  });
}

}  // namespace ibp
