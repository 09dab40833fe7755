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
#include "ibp_tile.h"

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

// ------------------------------------------------------------------ many rows

// A workgroup of WM x WN wavefronts computes 16 FM WM rows of A by 16 FN WN rows of B,
// operands staged in LDS through the direct global-to-LDS loads, two stages of which one
// is filled while the other is multiplied.  A stage holds 128 bytes of each row of A:
// 256 elements of e2m1 (two matrix instructions deep, instruction s takes blocks s,
// 2 + s, 4 + s, 6 + s) or 128 of e4m3 (one deep), and the same elements of B.
//
// LDS rows are 128 or 64 bytes; the 16-byte pieces of a row are permuted by the row
// number so that the 16 rows which a read takes at one piece fall into all 64 banks.
// The loads write LDS in lane order, so the permutation is made by the lanes' sources.
template <uint32_t PITCH> __device__ __forceinline__ uint32_t swizzle(uint32_t row, uint32_t piece) {
  return PITCH == 128 ? piece ^ ((row >> 1) & 7) : piece ^ ((row >> 2) & 3);
}

// One operand's part of a stage: ROWS rows of PITCH bytes of codes, their scale bytes.
template <uint32_t ROWS, uint32_t PITCH, uint32_t SCALES, uint32_t WAVES> struct Tile {
  static constexpr uint32_t kCodes = ROWS * PITCH, kBytes = kCodes + ROWS * SCALES;
  static constexpr uint32_t kLoads = kCodes / (1024 * WAVES);            // 16 bytes a lane
  static constexpr uint32_t kScaleLoads = (ROWS * SCALES / 4 + 64 * WAVES - 1) / (64 * WAVES);  // 4 bytes a lane

  const uint8_t *code[kLoads];
  uint32_t at[kLoads];
  const uint8_t *scale[kScaleLoads];
  uint32_t scale_at[kScaleLoads];

  __device__ __forceinline__ void init(const uint8_t *codes, const uint8_t *scales, uint64_t row0, uint64_t rows,
                                       uint32_t cp, uint32_t sp, uint32_t wave, uint32_t lane) {
#pragma unroll
    for (uint32_t i = 0; i < kLoads; ++i) {
      const uint32_t slot = (i * WAVES + wave) * 64 + lane, row = slot / (PITCH / 16);
      const uint64_t r = row0 + row < rows ? row0 + row : rows - 1;
      at[i] = swizzle<PITCH>(row, slot % (PITCH / 16)) * 16;
      code[i] = codes + r * cp;
    }
#pragma unroll
    for (uint32_t i = 0; i < kScaleLoads; ++i) {
      const uint32_t slot = (i * WAVES + wave) * 64 + lane, row = slot / (SCALES / 4);
      const uint64_t r = row0 + row < rows ? row0 + row : rows - 1;
      scale_at[i] = slot % (SCALES / 4) * 4;
      scale[i] = scales + r * sp;
    }
  }

  // Fills the tile with its rows' bytes from `k` (codes) and `b` (scales) on, zeros past the rows' ends.
  __device__ __forceinline__ void load(uint8_t *lds, uint32_t k, uint32_t cp, uint32_t b, uint32_t sp, uint32_t wave) {
#pragma unroll
    for (uint32_t i = 0; i < kLoads; ++i)
      to_lds16(k + at[i] < cp ? code[i] + k + at[i] : kZeros, lds + (i * WAVES + wave) * 1024);
#pragma unroll
    for (uint32_t i = 0; i < kScaleLoads; ++i)
      if ((i * WAVES + wave) * 256 < ROWS * SCALES)
        to_lds4(b + scale_at[i] < sp ? scale[i] + b + scale_at[i] : kZeros, lds + kCodes + (i * WAVES + wave) * 256);
  }
};

template <bool A8, int WM, int WN, int FM, int FN, int DO>
__global__ __launch_bounds__(WM *WN *64) void mx_tile_kernel(MxMatmulArgs a, uint32_t tiles_m, uint32_t tiles_n) {
  using TO = typename Num<DO>::T;
  constexpr uint32_t kWaves = WM * WN, kRowsA = 16 * FM * WM, kRowsB = 16 * FN * WN;
  constexpr uint32_t kPitchA = 128, kPitchB = A8 ? 64 : 128, kBlocks = A8 ? 4 : 8;
  constexpr int kDeep = A8 ? 1 : 2;
  using TileA = Tile<kRowsA, kPitchA, kBlocks, kWaves>;
  using TileB = Tile<kRowsB, kPitchB, kBlocks, kWaves>;
  constexpr uint32_t kStage = TileA::kBytes + TileB::kBytes;
  __shared__ __align__(1024) uint8_t stages[2 * kStage];
  const uint32_t lane = lane_id(), wave = uniform(threadIdx.x / kWave), r = lane & 15, g = lane >> 4;
  const TileId t = tile_of(blockIdx.x, tiles_m, tiles_n);
  const uint64_t m0 = (uint64_t)t.row * kRowsA, n0 = (uint64_t)t.col * kRowsB;

  const uint32_t nblk = (uint32_t)mx_blocks(a.K), sp = (uint32_t)mx_scale_pitch(a.K);
  const uint32_t cpa = (uint32_t)mx_code_pitch(a.K, A8), cpb = (uint32_t)mx_code_pitch(a.K, false);
  TileA ta;
  TileB tb;
  ta.init(a.a_codes, a.a_scales, m0, a.M, cpa, sp, wave, lane);
  tb.init(a.b_codes, a.b_scales, n0, a.N, cpb, sp, wave, lane);
  const uint32_t wm = (wave % WM) * 16 * FM, wn = (wave / WM) * 16 * FN;
  v4f acc[FN][FM];
#pragma unroll
  for (int n = 0; n < FN; ++n)
#pragma unroll
    for (int m = 0; m < FM; ++m) acc[n][m] = v4f{0, 0, 0, 0};

  const uint32_t steps = (nblk + kBlocks - 1) / kBlocks;
  auto fill = [&](uint8_t *st, uint32_t k) {
    ta.load(st, k * kPitchA, cpa, k * kBlocks, sp, wave);
    tb.load(st + TileA::kBytes, k * kPitchB, cpb, k * kBlocks, sp, wave);
  };
  auto multiply = [&](const uint8_t *st) {
    const uint8_t *sa = st, *sb = st + TileA::kBytes;
    int xs[FM], ws[FN];
#pragma unroll
    for (int m = 0; m < FM; ++m) {
      const uint8_t *p = sa + TileA::kCodes + (wm + 16 * m + r) * kBlocks + g * kDeep;
      xs[m] = A8 ? *p : *reinterpret_cast<const uint16_t *>(p);
    }
#pragma unroll
    for (int n = 0; n < FN; ++n) {
      const uint8_t *p = sb + TileB::kCodes + (wn + 16 * n + r) * kBlocks + g * kDeep;
      ws[n] = A8 ? *p : *reinterpret_cast<const uint16_t *>(p);
    }
    const uint4 none = make_uint4(0u, 0u, 0u, 0u);
#pragma unroll
    for (int d = 0; d < kDeep; ++d) {
      v8i w[FN];
#pragma unroll
      for (int n = 0; n < FN; ++n) {
        const uint32_t row = wn + 16 * n + r;
        w[n] = operand(*reinterpret_cast<const uint4 *>(sb + row * kPitchB + swizzle<kPitchB>(row, g * kDeep + d) * 16), none);
      }
#pragma unroll
      for (int m = 0; m < FM; ++m) {
        const uint32_t row = wm + 16 * m + r;
        v8i v;
        if constexpr (A8)
          v = operand(*reinterpret_cast<const uint4 *>(sa + row * kPitchA + swizzle<kPitchA>(row, g) * 16),
                      *reinterpret_cast<const uint4 *>(sa + row * kPitchA + swizzle<kPitchA>(row, 4 + g) * 16));
        else
          v = operand(*reinterpret_cast<const uint4 *>(sa + row * kPitchA + swizzle<kPitchA>(row, g * 2 + d) * 16), none);
#pragma unroll
        for (int n = 0; n < FN; ++n) acc[n][m] = mfma_mx<A8>(w[n], v, acc[n][m], ws[n], xs[m], d);
      }
    }
  };
  // The two stages do not overlap; __restrict__ says so to the compiler, which otherwise
  // would wait for the loads in flight before every LDS read.
  auto both = [&](uint8_t *__restrict__ next, const uint8_t *__restrict__ now, uint32_t k) {
    if (k < steps) fill(next, k);
    multiply(now);
  };
  // the loads of a stage are waited for, then all wavefronts know that it is full and that the other is free
  auto ready = [&] {
    __builtin_amdgcn_s_waitcnt(kWaitVmcnt0);
    __syncthreads();
  };
  if (steps) fill(stages, 0);
#pragma unroll 1
  for (uint32_t k = 0; k < steps; ++k) {
    ready();
    both(stages + ((k + 1) & 1) * kStage, stages + (k & 1) * kStage, k + 1);
  }
  TO *y = static_cast<TO *>(a.y);
#pragma unroll
  for (int m = 0; m < FM; ++m) {
    const uint64_t row = m0 + wm + 16 * m + r;
    if (row >= a.M) continue;
#pragma unroll
    for (int n = 0; n < FN; ++n) store4<TO>(y + row * a.N, n0 + wn + 16 * n + 4 * g, a.N, acc[n][m]);
  }
}

template <bool A8, int WM, int WN, int FM, int FN> hipError_t go_tile(const MxMatmulArgs &a, hipStream_t s) {
  const uint64_t tm = (a.M + 16 * FM * WM - 1) / (16 * FM * WM), tn = (a.N + 16 * FN * WN - 1) / (16 * FN * WN);
  if (tm * tn > 0x3FFFFF) return hipErrorInvalidValue;
  return with_dtype(a.dtype, [&](auto d) {
    mx_tile_kernel<A8, WM, WN, FM, FN, d.value>
        <<<(uint32_t)(tm * tn), WM * WN * kWave, 0, s>>>(a, (uint32_t)tm, (uint32_t)tn);
    return hipGetLastError();
  });
}

template <bool A8> hipError_t go(const MxMatmulArgs &a, hipStream_t s) {
  const uint64_t big = ((a.M + 255) / 256) * ((a.N + 255) / 256), mid = ((a.M + 127) / 128) * ((a.N + 127) / 128);
  if (a.M <= 16) return go_direct<A8, 1>(a, s);
  if (big >= 192) return go_tile<A8, 2, 4, 8, 4>(a, s);
  if (mid >= 64) return go_tile<A8, 2, 2, 4, 4>(a, s);
  return go_direct<A8, 4>(a, s);
}

}  // namespace

uint64_t mx_matmul_workspace(uint64_t, uint64_t, uint32_t, bool) { return 0; }

hipError_t launch_mx_matmul(const MxMatmulArgs &a, hipStream_t s) {
  return a.a_e4m3 ? go<true>(a, s) : go<false>(a, s);
}

}  // namespace ibp
