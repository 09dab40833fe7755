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
#include "ibp_tile.h"

namespace ibp {
namespace {

using namespace dev;

typedef short v4s __attribute__((ext_vector_type(4)));
typedef __bf16 v8b __attribute__((ext_vector_type(8)));

constexpr uint32_t kT = 64;  // tokens per stage

// LDS byte of the 16-byte piece `c16` of row t of a tile of W columns.  The 32-byte
// pieces of a row are permuted by the low bits of t: a transposing read takes 32 bytes
// of each of eight rows at a time, which then fall into all 64 banks.
template <uint32_t W> __device__ __forceinline__ uint32_t tile_at(uint32_t t, uint32_t c16) {
  return t * (W * 2) + ((((c16 >> 1) ^ (t & 7)) << 5) | ((c16 & 1) << 4));
}

// Eight BF16 of column block `col` (16 columns) of 32 rows from `t0` on, in the order of
// the matrix instruction's k: lane group g takes rows 4 g .. 4 g + 3 and 16 + 4 g ..
// 16 + 4 g + 3; both operands do, so the sum is over the same tokens.
template <uint32_t W> __device__ __forceinline__ v8b fragment(const uint8_t *tile, uint32_t t0, uint32_t col, uint32_t lane) {
  const uint32_t t = (lane >> 4) * 4 + ((lane & 15) >> 2), sub = (lane & 3) * 8;
  const uint8_t *at = tile + (t0 + t) * (W * 2) + ((col ^ (t & 7)) << 5) + sub;
  using L = __attribute__((address_space(3))) v4s;
  const v4s lo = __builtin_amdgcn_ds_read_tr16_b64_v4i16((L *)at);
  const v4s hi = __builtin_amdgcn_ds_read_tr16_b64_v4i16((L *)(at + 16 * W * 2));
  return __builtin_bit_cast(v8b, __builtin_shufflevector(lo, hi, 0, 1, 2, 3, 4, 5, 6, 7));
}

// Eight e4m3 codes of one block as BF16, exactly.
__device__ __forceinline__ v8b decode8(uint2 q, float f) {
  typedef __bf16 v2b __attribute__((ext_vector_type(2)));
  const v2b a = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(q.x, f, false);
  const v2b b = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(q.x, f, true);
  const v2b c = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(q.y, f, false);
  const v2b d = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(q.y, f, true);
  return v8b{a[0], a[1], b[0], b[1], c[0], c[1], d[0], d[1]};
}

// A workgroup of WI x WO wavefronts computes 16 FI WI (i) by 16 FO WO (o) elements of dW
// over the tokens [z * t_each, (z + 1) * t_each), z = blockIdx.y, into dst + z * N * K.
// Two stages in LDS: while one is multiplied, the other's dY comes by direct
// global-to-LDS loads (DIRECT: rows of dY aligned to 16 bytes) and its X through
// registers, where it is decoded.
template <int WI, int WO, int FI, int FO, bool DIRECT, int DO>
__global__ __launch_bounds__(WI *WO *64) void wgrad_kernel(MxWgradArgs a, void *dst, uint64_t t_each, uint32_t tiles_o,
                                                           uint32_t tiles_i) {
  using TO = typename Num<DO>::T;
  constexpr uint32_t kWaves = WI * WO, kThreads = kWaves * 64, kWideI = 16 * FI * WI, kWideO = 16 * FO * WO;
  constexpr uint32_t kPiecesY = kT * kWideO / 8 / kThreads, kPiecesX = kT * kWideI / 8 / kThreads;
  constexpr uint32_t kBytesY = kT * kWideO * 2, kStage = kBytesY + kT * kWideI * 2;
  __shared__ __align__(1024) uint8_t stages[2 * kStage];
  const uint32_t lane = lane_id(), wave = uniform(threadIdx.x / kWave);
  const TileId tile = tile_of(blockIdx.x, tiles_o, tiles_i);
  const uint32_t o0 = tile.row * kWideO, i0 = tile.col * kWideI;
  const uint32_t wi = (wave % WI) * FI, wo = (wave / WI) * FO;  // in blocks of 16
  const uint64_t t0 = blockIdx.y * t_each, t1 = t0 + t_each < a.T ? t0 + t_each : a.T;
  const uint32_t cp = (uint32_t)mx_code_pitch(a.K, true), sp = (uint32_t)mx_scale_pitch(a.K);
  const __bf16 *dy = static_cast<const __bf16 *>(a.dy);

  v4f acc[FI][FO];
#pragma unroll
  for (int x = 0; x < FI; ++x)
#pragma unroll
    for (int y = 0; y < FO; ++y) acc[x][y] = v4f{0, 0, 0, 0};

  uint2 qx[kPiecesX];
  uint32_t sx[kPiecesX];
  Vec8<__bf16> vy[DIRECT ? 1 : kPiecesY];
  // starts the loads of the stage that begins at token tb
  auto fetch = [&](uint8_t *st, uint64_t tb) {
#pragma unroll
    for (uint32_t p = 0; p < kPiecesY; ++p) {
      // LDS takes the pieces in lane order; the permutation is made by their sources
      const uint32_t slot = p * kThreads + threadIdx.x, t = slot / (kWideO / 8), s16 = slot % (kWideO / 8);
      const uint32_t c = o0 + ((((s16 >> 1) ^ (t & 7)) << 1) | (s16 & 1)) * 8;
      if constexpr (DIRECT)
        to_lds16(tb + t < t1 && c < a.N ? reinterpret_cast<const uint8_t *>(dy + (tb + t) * a.N + c) : kZeros,
                 st + (p * kWaves + wave) * 1024);
      else
        vy[p] = load8<__bf16>(dy + (tb + t < t1 ? tb + t : t1 - 1) * a.N, c, a.N);
    }
#pragma unroll
    for (uint32_t p = 0; p < kPiecesX; ++p) {
      const uint32_t slot = p * kThreads + threadIdx.x, t = slot / (kWideI / 8), c = i0 + slot % (kWideI / 8) * 8;
      const bool in = tb + t < t1 && c < cp;
      qx[p] = in ? *reinterpret_cast<const uint2 *>(a.x_codes + (tb + t) * cp + c) : make_uint2(0u, 0u);
      sx[p] = in ? a.x_scales[(tb + t) * sp + c / kMxBlock] : 127u;
    }
  };
  // what came through registers goes to LDS
  auto settle = [&](uint8_t *st, uint64_t tb) {
    if constexpr (!DIRECT) {
#pragma unroll
      for (uint32_t p = 0; p < kPiecesY; ++p) {
        const uint32_t slot = p * kThreads + threadIdx.x, t = slot / (kWideO / 8), s16 = slot % (kWideO / 8);
        const uint32_t c = o0 + ((((s16 >> 1) ^ (t & 7)) << 1) | (s16 & 1)) * 8;
        *reinterpret_cast<v8b *>(st + slot * 16) = (v8b)settle8<__bf16>(vy[p], tb + t < t1 ? c : a.N, a.N);
      }
    }
#pragma unroll
    for (uint32_t p = 0; p < kPiecesX; ++p) {
      const uint32_t slot = p * kThreads + threadIdx.x, t = slot / (kWideI / 8), c16 = slot % (kWideI / 8);
      *reinterpret_cast<v8b *>(st + kBytesY + tile_at<kWideI>(t, c16)) = decode8(qx[p], mx_factor(sx[p]));
    }
  };
  auto multiply = [&](const uint8_t *st) {
#pragma unroll
    for (uint32_t t = 0; t < kT; t += 32) {
      v8b fy[FO];
#pragma unroll
      for (int y = 0; y < FO; ++y) fy[y] = fragment<kWideO>(st, t, wo + y, lane);
#pragma unroll
      for (int x = 0; x < FI; ++x) {
        const v8b fx = fragment<kWideI>(st + kBytesY, t, wi + x, lane);
#pragma unroll
        for (int y = 0; y < FO; ++y) acc[x][y] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(fx, fy[y], acc[x][y], 0, 0, 0);
      }
    }
  };
  // the stages do not overlap, which __restrict__ tells the compiler: it would wait for
  // the loads in flight before every LDS read
  auto both = [&](uint8_t *__restrict__ next, const uint8_t *__restrict__ now, uint64_t tb) {
    if (tb < t1) fetch(next, tb);
    multiply(now);
    if (tb < t1) settle(next, tb);
  };
  uint32_t cur = 0;
  if (t0 < t1) {
    fetch(stages, t0);
    settle(stages, t0);
  }
#pragma unroll 1
  for (uint64_t tb = t0; tb < t1; tb += kT) {
    __builtin_amdgcn_s_waitcnt(kWaitVmcnt0);  // the direct loads of the stage
    __syncthreads();
    both(stages + (cur ^ 1) * kStage, stages + cur * kStage, tb + kT);
    cur ^= 1;
  }
  // a lane has four consecutive i of one o
  TO *dw = static_cast<TO *>(dst) + (uint64_t)blockIdx.y * a.N * a.K;
#pragma unroll
  for (int y = 0; y < FO; ++y) {
    const uint32_t o = o0 + (wo + y) * 16 + (lane & 15);
    if (o >= a.N) continue;
#pragma unroll
    for (int x = 0; x < FI; ++x) store4<TO>(dw + (uint64_t)o * a.K, i0 + (wi + x) * 16 + 4 * (lane >> 4), a.K, acc[x][y]);
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

// Tile and ranges of tokens.  256 x 256 tiles read each operand half as often as 128 x
// 128 ones, so they are taken where tiles and tokens give every CU 512 tokens of one
// (16384 tokens: 2048 x 2048 171 us against 227, 512 x 512 42 against 36).  The tokens are
// cut into ranges until there is a workgroup per CU (16384 tokens of 1024 x 1024: 556 us
// in one range, 64 in sixteen): each range's sums are written and read once in 32 bits.
struct Plan {
  bool big;
  uint32_t tiles_o, tiles_i;
  uint32_t splits;
  uint64_t t_each;
};

Plan plan_of(uint64_t T, uint32_t N, uint32_t K) {
  Plan p;
  const uint64_t big = (((uint64_t)N + 255) / 256) * (((uint64_t)K + 255) / 256);
  p.big = big * ((T + 511) / 512) >= 256;
  const uint32_t wide = p.big ? 256 : 128;
  p.tiles_o = (uint32_t)(((uint64_t)N + wide - 1) / wide);
  p.tiles_i = (uint32_t)(((uint64_t)K + wide - 1) / wide);
  const uint64_t tiles = (uint64_t)p.tiles_o * p.tiles_i, least = p.big ? 512 : 128;
  const uint64_t want = 256 / tiles, most = (T + least - 1) / least;
  uint64_t n = want < most ? want : most;
  n = n < 1 ? 1 : (n > 32 ? 32 : n);
  p.t_each = ((T + n - 1) / n + kT - 1) / kT * kT;
  if (p.t_each == 0) p.t_each = kT;
  p.splits = T ? (uint32_t)((T + p.t_each - 1) / p.t_each) : 1;
  return p;
}

template <int DO> hipError_t go(const MxWgradArgs &a, const Plan &p, void *dst, hipStream_t s) {
  const bool direct = a.N % 8 == 0 && (uintptr_t)a.dy % 16 == 0;
  const dim3 grid(p.tiles_o * p.tiles_i, p.splits);
  if (p.big && direct)
    wgrad_kernel<2, 4, 8, 4, true, DO><<<grid, 512, 0, s>>>(a, dst, p.t_each, p.tiles_o, p.tiles_i);
  else if (p.big)
    wgrad_kernel<2, 4, 8, 4, false, DO><<<grid, 512, 0, s>>>(a, dst, p.t_each, p.tiles_o, p.tiles_i);
  else if (direct)
    wgrad_kernel<2, 2, 4, 4, true, DO><<<grid, 256, 0, s>>>(a, dst, p.t_each, p.tiles_o, p.tiles_i);
  else
    wgrad_kernel<2, 2, 4, 4, false, DO><<<grid, 256, 0, s>>>(a, dst, p.t_each, p.tiles_o, p.tiles_i);
  return hipGetLastError();
}

}  // namespace

uint64_t mx_wgrad_workspace(uint64_t T, uint32_t N, uint32_t K) {
  const Plan p = plan_of(T, N, K);
  return p.splits > 1 ? (uint64_t)p.splits * N * K * 4 : 0;
}

hipError_t launch_mx_wgrad(const MxWgradArgs &a, hipStream_t s) {
  const Plan p = plan_of(a.T, a.N, a.K);
  if (p.splits > 1) {
    const hipError_t e = go<IBP_F32>(a, p, a.ws, s);
    if (e != hipSuccess) return e;
  }
  return with_dtype(a.dtype, [&](auto d) {
    if (p.splits == 1) return go<d.value>(a, p, a.dw, s);
    const uint64_t n = ((uint64_t)a.N * a.K + kBlock * 4 - 1) / (kBlock * 4);
    wgrad_join_kernel<d.value><<<(uint32_t)(n < 4096 ? n : 4096), kBlock, 0, s>>>(a, p.splits);
    return hipGetLastError();
  });
}

}  // namespace ibp
