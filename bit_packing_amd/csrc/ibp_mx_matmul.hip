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

// Scales are the low bytes of ws and xs; format codes: 0 e4m3, 4 e2m1.
//
// Within a block the instruction adds products aligned to the largest and drops what lies
// more than 13 binary places below it, counted by the factors' exponents (measured:
// 256 * 1 + 2^-5 * 1 is kept, + 2^-6 is not; 448 * 6 + 2.25 * 0.5, whose last bit is 2^-3, is
// kept whole).  Products of e2m1 fit (4 * 4 down to 1/4), sums over blocks are 32-bit.
// Products of e4m3 span 20 places (256 * 4 down to 2^-10), so its elements of magnitude 2 and
// more, whose codes have bit 6, go through one instruction (2^10 down to 2^-3) and the rest
// through another (4 down to 2^-10): nothing is dropped.  In one instruction a block whose
// large products cancel, as those of an outlier column may, would lose its result: 8192 x
// 8192 x 8192 would take 370 us so, against 600.
//
// split takes the large elements' bytes out of four.
__device__ __forceinline__ int split(int &x) {
  // bytes with the bit: a selector of 12 gives 0x00, a larger one 0xFF
  const int mask = (int)__builtin_amdgcn_perm(0u, 0u, ((uint32_t)x & 0x40404040u) | 0x0C0C0C0Cu);
  const int high = x & mask;
  x &= ~mask;
  return high;
}

template <bool A8> __device__ __forceinline__ v4f mfma_one(v8i w, v8i x, v4f acc, int ws, int xs) {
  return __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(w, x, acc, 4, A8 ? 0 : 4, 0, ws, 0, xs);
}

template <bool A8> __device__ __forceinline__ v4f mfma_mx(v8i w, v8i x, v4f acc, int ws, int xs) {
  if constexpr (A8) {
    v8i high;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      int low = x[i];
      high[i] = split(low);
      x[i] = low;
    }
    acc = mfma_one<A8>(w, high, acc, ws, xs);
  }
  return mfma_one<A8>(w, x, acc, ws, xs);
}

__device__ __forceinline__ v8i operand(uint4 lo, uint4 hi) {
  return v8i{(int)lo.x, (int)lo.y, (int)lo.z, (int)lo.w, (int)hi.x, (int)hi.y, (int)hi.z, (int)hi.w};
}

// 16 scale bytes of a row from block b on, zeros past its end.
__device__ __forceinline__ uint4 scales16(const uint8_t *row, uint32_t b, uint32_t pitch) {
  typedef uint32_t V __attribute__((ext_vector_type(4), aligned(4)));
  V v = {};
  if (b + 16 <= pitch) {
    v = *reinterpret_cast<const V *>(row + b);
  } else {
#pragma unroll
    for (uint32_t j = 0; j < 4; ++j)
      if (b + 4 * j < pitch) v[j] = *reinterpret_cast<const uint32_t *>(row + b + 4 * j);
  }
  return make_uint4(v[0], v[1], v[2], v[3]);
}

// Few rows of A: bound by the latency of a step's loads, of which the next step's are not in
// flight (1 x 8192 outputs, 8192 deep: 8.3 us from e2m1, 4.3 TB/s of weights, 10.2 from e4m3, 3.5
// TB/s; half of the wavefronts' time is waiting).  A workgroup computes 16 x 16 outputs, its
// wavefronts take the steps of k in turn and their sums are added in order through LDS.  A step
// is 16 blocks, four matrix instructions; each load takes 64 consecutive bytes of 16 rows.
//
// GROUPED: the rows are sorted by expert, and blockIdx.y counts units of 16 rows of one
// expert, as many as there can be; those that there are not have nothing to do.
template <bool GROUPED, bool A8, int DO> __global__ void mx_direct_kernel(MxMatmulArgs a) {
  using TO = typename Num<DO>::T;
  extern __shared__ float red[];
  const uint32_t lane = lane_id(), wave = uniform(threadIdx.x / kWave), waves = blockDim.x / kWave;
  const uint32_t r = lane & 15, g = lane >> 4;
  const uint64_t n0 = (uint64_t)blockIdx.x * 16;
  uint64_t m0 = (uint64_t)blockIdx.y * 16;
  if constexpr (GROUPED) {
    const Experts x{a.offsets, a.experts, 4, a.M};
    if (a.err && blockIdx.x == 0 && blockIdx.y == 0 && wave == 0) check_offsets(x, a.err);
    const UnitSearch<false> search(x);
    if (blockIdx.y >= search.total) return;
    const Unit u = search.find(blockIdx.y);
    if (u.row0 >= u.end) return;
    m0 = u.row0;
    a.M = u.end;
    a.b_codes += u.expert * a.N * mx_code_pitch(a.K, false);
    a.b_scales += u.expert * a.N * mx_scale_pitch(a.K);
  }
  const uint32_t nblk = (uint32_t)mx_blocks(a.K), sp = (uint32_t)mx_scale_pitch(a.K);
  const uint32_t wp = (uint32_t)mx_code_pitch(a.K, false), xp = (uint32_t)mx_code_pitch(a.K, A8);
  // rows past the end repeat the last one; their results are not stored
  const uint64_t n = n0 + r < a.N ? n0 + r : a.N - 1, m = m0 + r < a.M ? m0 + r : a.M - 1;
  const uint8_t *wc = a.b_codes + n * wp, *wsc = a.b_scales + n * sp;
  const uint8_t *xc = a.a_codes + m * xp, *xsc = a.a_scales + m * sp;
  v4f acc{0, 0, 0, 0};
  for (uint32_t b0 = wave * kStep; b0 < nblk; b0 += waves * kStep) {
    uint4 w[4], lo[4], hi[4];
#pragma unroll
    for (int s = 0; s < 4; ++s) w[s] = piece(wc, (b0 + 4 * s + g) * 16, wp);
    const uint4 ws4 = scales16(wsc, b0, sp), xs4 = scales16(xsc, b0, sp);
#pragma unroll
    for (int s = 0; s < 4; ++s) {
      lo[s] = piece(xc, A8 ? (b0 + 4 * s) * 32 + 16 * g : (b0 + 4 * s + g) * 16, xp);
      hi[s] = A8 ? piece(xc, (b0 + 4 * s) * 32 + 64 + 16 * g, xp) : make_uint4(0u, 0u, 0u, 0u);
    }
    const uint32_t wd[4] = {ws4.x, ws4.y, ws4.z, ws4.w}, xd[4] = {xs4.x, xs4.y, xs4.z, xs4.w};
#pragma unroll
    for (int s = 0; s < 4; ++s)
      acc = mfma_mx<A8>(operand(w[s], make_uint4(0u, 0u, 0u, 0u)), operand(lo[s], hi[s]), acc, (int)(wd[s] >> (8 * g)),
                         (int)(xd[s] >> (8 * g)));
  }
  if (waves > 1) {
    if (wave) *reinterpret_cast<v4f *>(red + (wave - 1) * 256 + lane * 4) = acc;
    __syncthreads();
    if (wave) return;
    for (uint32_t k = 0; k + 1 < waves; ++k) acc += *reinterpret_cast<const v4f *>(red + k * 256 + lane * 4);
  }
  if (m0 + r < a.M) store4<TO>(static_cast<TO *>(a.y) + (m0 + r) * a.N, n0 + 4 * g, a.N, acc);
}

template <bool A8> hipError_t go_direct(const MxMatmulArgs &a, hipStream_t s) {
  const uint64_t gx = (a.N + 15) / 16, gy = (a.M + 15) / 16;
  const uint32_t steps = (uint32_t)((mx_blocks(a.K) + kStep - 1) / kStep);
  // Up to one workgroup a CU sixteen wavefronts, which share a long k; beyond, four (8192 deep,
  // one row of e4m3: 4096 outputs 6.6 us against 8.1, 4624 outputs 10.9 against 9.5, 8176 11.2
  // against 9.7; of e2m1 5.8 against 6.4, 8.7 against 8.2, 8.8 against 8.3).
  uint32_t waves = gx * gy <= 256 ? 16 : 4;
  while (waves > 1 && waves > steps) waves /= 2;
  return with_dtype(a.dtype, [&](auto d) {
    mx_direct_kernel<false, A8, d.value><<<dim3((uint32_t)gx, (uint32_t)gy), waves * kWave, (waves - 1) * 1024, s>>>(a);
    return hipGetLastError();
  });
}

// ------------------------------------------------------------------ many rows

// A workgroup of WM x WN wavefronts computes 16 FM WM rows of A by 16 FN WN rows of B over
// stages_each stages of k, from blockIdx.y * stages_each on, into dst + blockIdx.y * M * N.
// Operands go through LDS by the direct global-to-LDS loads, in stages of 128 elements
// of every row, one matrix instruction deep, in a ring of kStages: while one is
// multiplied the loads of the next ones are in flight.  8192 x 8192 x 8192 in e2m1 takes
// 272 us, 4.0 PFLOP/s (310 us with two stages of 256 elements and all wavefronts in step);
// with the loads left out 80% of that, with the matrix instructions left out as long: it
// is bound by a turn's two phases, reading LDS and issuing loads in one, multiplying in
// the other, and by power: the clock falls to 2.0 GHz.  The 32 x 32 x 64 matrix instruction
// takes 2% fewer cycles at a clock 5% lower (with packing 330 us against 320); without
// phases, reading each fragment's successor once it is used, 331 against 327.
// LDS rows are 128 (e4m3) or 64 bytes (e2m1).
//
// GROUPED: the tiles are cut from each expert's rows.  Their number is on the device, the
// workgroups are as many as it can be; those beyond it have nothing to do.
template <bool GROUPED, bool A8, int WM, int WN, int FM, int FN, int DO>
__global__ __launch_bounds__(WM *WN *64) void mx_tile_kernel(MxMatmulArgs a, void *dst, uint32_t tiles_m,
                                                             uint32_t tiles_n, uint32_t stages_each) {
  using TO = typename Num<DO>::T;
  constexpr uint32_t kWaves = WM * WN, kRowsA = 16 * FM * WM, kRowsB = 16 * FN * WN;
  constexpr uint32_t kPitchA = A8 ? 128 : 64, kPitchB = 64, kBlocks = 4;
  using TileA = Tile<kRowsA, kPitchA, kWaves>;
  using TileB = Tile<kRowsB, kPitchB, kWaves>;
  static_assert(kRowsA + kRowsB == 64 * kWaves, "a wavefront loads the scales of 64 rows");
  constexpr uint32_t kStage = TileA::kBytes + TileB::kBytes, kStages = A8 ? 3 : 4;
  constexpr uint32_t kLoads = TileA::kLoads + TileB::kLoads;  // a wavefront's loads per stage
  // Scales come for kGroup stages at a time, 16 bytes of each row of A, then of B: a dword
  // a stage would ask L2 for a line per row and stage, as many requests as the codes.
  constexpr uint32_t kGroup = 4, kRows = kRowsA + kRowsB, kScales = kRows * 16;
  static_assert(kStages * kStage + 2 * kScales <= 160 * 1024 && (kStages - 2) * kLoads < 16, "");
  __shared__ __align__(1024) uint8_t ring[kStages * kStage + 2 * kScales];
  const uint32_t lane = lane_id(), wave = uniform(threadIdx.x / kWave), r = lane & 15, g = lane >> 4;
  const uint64_t all_m = a.M;
  uint64_t m0, n0;
  if constexpr (GROUPED) {
    static_assert((kRowsA & (kRowsA - 1)) == 0, "");
    const Experts x{a.offsets, a.experts, (uint32_t)__builtin_ctz(kRowsA), a.M};
    if (a.err && blockIdx.x == 0 && blockIdx.y == 0 && wave == 0) check_offsets(x, a.err);
    const UnitSearch<false> search(x);
    if (blockIdx.x >= (uint64_t)search.total * tiles_n) return;
    const TileId t = tile_of(blockIdx.x, search.total, tiles_n);
    const Unit u = search.find(t.row);
    if (u.row0 >= u.end) return;
    m0 = u.row0;
    n0 = (uint64_t)t.col * kRowsB;
    a.M = u.end;
    a.b_codes += u.expert * a.N * mx_code_pitch(a.K, false);
    a.b_scales += u.expert * a.N * mx_scale_pitch(a.K);
  } else {
    const TileId t = tile_of(blockIdx.x, tiles_m, tiles_n);
    m0 = (uint64_t)t.row * kRowsA;
    n0 = (uint64_t)t.col * kRowsB;
  }

  const uint32_t nblk = (uint32_t)mx_blocks(a.K), sp = (uint32_t)mx_scale_pitch(a.K);
  const uint32_t cpa = (uint32_t)mx_code_pitch(a.K, A8), cpb = (uint32_t)mx_code_pitch(a.K, false);
  TileA ta;
  TileB tb;
  ta.init(a.a_codes, m0, a.M, cpa, wave, lane);
  tb.init(a.b_codes, n0, a.N, cpb, wave, lane);
  const uint8_t *scale;
  {
    const uint32_t row = wave * 64 + lane;
    const bool of_a = row < kRowsA;
    const uint64_t at = of_a ? m0 + row : n0 + row - kRowsA, rows = of_a ? a.M : a.N;
    scale = (of_a ? a.a_scales : a.b_scales) + (at < rows ? at : rows - 1) * sp;
  }
  const uint32_t wm = (wave % WM) * 16 * FM, wn = (wave / WM) * 16 * FN;
  v4f acc[FN][FM];
#pragma unroll
  for (int n = 0; n < FN; ++n)
#pragma unroll
    for (int m = 0; m < FM; ++m) acc[n][m] = v4f{0, 0, 0, 0};

  // stages of this workgroup's range of k, which begins at a whole group of scales
  const uint32_t all = (nblk + kBlocks - 1) / kBlocks, begin = blockIdx.y * stages_each;
  const uint32_t steps = all - begin < stages_each ? all - begin : stages_each;
  // Always kLoads loads, of zeros past the rows' end: the waits below count on it.
  auto fill = [&](uint8_t *st, uint32_t stage) {
    const uint32_t k = begin + stage;
    ta.load(st, k * kPitchA, cpa, wave);
    tb.load(st + TileA::kBytes, k * kPitchB, cpb, wave);
  };
  // Scales of group q, 16 bytes a row; where the rows end inside, their last dwords come
  // through registers with zeros after them (a neighbour's scale may be NaN).
  auto fill_scales = [&](uint8_t *sc, uint32_t group) {
    const uint32_t q = begin / kGroup + group;
    if ((q + 1) * 16 <= sp) {
      to_lds16(scale + q * 16, sc + wave * 1024);
    } else {
      uint32_t d[kGroup];
#pragma unroll
      for (uint32_t j = 0; j < kGroup; ++j)
        d[j] = q * 16 + j * 4 < sp ? *reinterpret_cast<const uint32_t *>(scale + q * 16 + j * 4) : 0u;
      *reinterpret_cast<uint4 *>(sc + wave * 1024 + lane * 16) = make_uint4(d[0], d[1], d[2], d[3]);
    }
  };
  v8i w[FN], v[FM];
  int ws[FN], xs[FM];
  // a fragment's rows are 16 apart and its permutation goes by r alone: one address, then offsets
  const uint32_t at_a = (wm + r) * kPitchA + swizzle<kPitchA>(r, g) * 16;
  const uint32_t at_a2 = (wm + r) * kPitchA + swizzle<kPitchA>(r, 4 + g) * 16;  // e4m3: blocks 2 and 3
  const uint32_t at_b = (wn + r) * kPitchB + swizzle<kPitchB>(r, g) * 16;
  auto read = [&](const uint8_t *st, const uint8_t *sc) {
    const uint4 none = make_uint4(0u, 0u, 0u, 0u);
#pragma unroll
    for (int n = 0; n < FN; ++n) {
      w[n] = operand(*reinterpret_cast<const uint4 *>(st + TileA::kBytes + at_b + n * 16 * kPitchB), none);
      ws[n] = sc[(kRowsA + wn + r) * 16 + g + n * 256];
    }
#pragma unroll
    for (int m = 0; m < FM; ++m) {
      v[m] = operand(*reinterpret_cast<const uint4 *>(st + at_a + m * 16 * kPitchA),
                     A8 ? *reinterpret_cast<const uint4 *>(st + at_a2 + m * 16 * kPitchA) : none);
      xs[m] = sc[(wm + r) * 16 + g + m * 256];
    }
  };
  uint8_t *const scales = ring + kStages * kStage;
  // Each turn of the loop is a reading phase and a multiplying phase with a barrier after
  // each.  With two wavefronts a SIMD the second half of the wavefronts runs one phase
  // behind the first (kPingPong), so LDS serves one half while the other multiplies; in
  // step, all would read at once and the matrix units idle meanwhile.  With four stages
  // the loads are issued between the matrix instructions (they cost the reading phase,
  // the longer one, a third of its time); with three they would come too late there.
  constexpr bool kPingPong = kWaves == 8, kLateFill = kStages >= 4;
  const bool behind = kPingPong && wave >= kWaves / 2;
  // What is filled is not what is read; __restrict__ says so to the compiler, which
  // otherwise would wait for all loads in flight before an LDS read.
  auto load_phase = [&](uint8_t *__restrict__ next, uint8_t *__restrict__ next_scales, const uint8_t *__restrict__ now,
                        const uint8_t *__restrict__ now_scales, uint32_t k) {
    if (!kLateFill) fill(next, k + kStages - 1);
    if (k % kGroup == 0) fill_scales(next_scales, k / kGroup + 1);
    read(now, now_scales);
  };
#pragma unroll
  for (uint32_t k = 0; k + 1 < kStages; ++k) fill(ring + k * kStage, k);
  fill_scales(scales, 0);
  __builtin_amdgcn_s_waitcnt(kWaitVmcnt0 & ~0x0F00);  // and LDS writes
  phase_barrier();
  if (behind) phase_barrier();
  uint32_t now = 0, next = kStages - 1;  // ring places of stage k and of stage k - 1, which is filled anew
#pragma unroll 1
  for (uint32_t k = 0; k < steps; ++k) {
    const uint32_t odd = k / kGroup & 1;
    uint8_t *const free_stage = ring + next * kStage;
    load_phase(free_stage, scales + (odd ^ 1) * kScales, ring + now * kStage, scales + odd * kScales + k % kGroup * 4, k);
    next = now;
    now = now + 1 == kStages ? 0 : now + 1;
    // These reads are done, and this wavefront's loads of stage k + 1 (not those of the stages
    // after it; loads of scales in between make the wait longer, never shorter, and are
    // kGroup stages early): after one or two barriers the first half reads it.
    __builtin_amdgcn_s_waitcnt(0x0070 | (kStages - (kLateFill ? 3 : 2)) * kLoads);
    phase_barrier();
    __builtin_amdgcn_s_setprio(1);
    if constexpr (A8) {
      // A fragment's successor is split between its matrix instructions, four bytes at a time,
      // which they hide: split all at once, before them, the matrix units would wait meanwhile
      // (8192 x 8192 x 8192: 740 us, and 727 with few fragments a wavefront, against 600).
      v8i high, next;
      constexpr int kEach = 2 * FN / 8;  // matrix instructions for four bytes
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        int low = v[0][i];
        high[i] = split(low);
        v[0][i] = low;
      }
#pragma unroll
      for (int m = 0; m < FM; ++m) {
#pragma unroll
        for (int i = 0; i < 2 * FN; ++i) {
          const int n = i % FN;
          acc[n][m] = mfma_one<A8>(w[n], i < FN ? high : v[m], acc[n][m], ws[n], xs[m]);
          if (m + 1 < FM && i % kEach == 0) {
            int low = v[m + 1 < FM ? m + 1 : 0][i / kEach];
            next[i / kEach] = split(low);
            v[m + 1 < FM ? m + 1 : 0][i / kEach] = low;
          }
          __builtin_amdgcn_sched_barrier(0);
        }
        high = next;
      }
    } else {
#pragma unroll
      for (int m = 0; m < FM; ++m) {
#pragma unroll
        for (int n = 0; n < FN; ++n) acc[n][m] = mfma_one<A8>(w[n], v[m], acc[n][m], ws[n], xs[m]);
        if (kLateFill && m == 0) {
          __builtin_amdgcn_sched_barrier(0);  // the compiler would issue the loads first
          fill(free_stage, k + kStages - 1);
        }
      }
    }
    __builtin_amdgcn_sched_barrier(0);
    __builtin_amdgcn_s_setprio(0);
    phase_barrier();
  }
  if (kPingPong && wave < kWaves / 2) phase_barrier();
  __builtin_amdgcn_s_waitcnt(kWaitVmcnt0);  // no load into LDS outlives the workgroup
  __syncthreads();
  static_assert(kWaves * out_bytes<TO, FN>() <= sizeof(ring), "");
  store_fragments<TO, FM, FN, 2, GROUPED>(reinterpret_cast<TO *>(ring + wave * out_bytes<TO, FN>()),
                              static_cast<TO *>(dst) + (uint64_t)blockIdx.y * all_m * a.N, (uint32_t)(m0 + wm), (uint32_t)a.M,
                              (uint32_t)(n0 + wn), (uint32_t)a.N, lane,
                              [&](int m, int n) { return acc[n][m]; });
}

// Adds the ranges' sums in order.
template <int DO> __global__ __launch_bounds__(kBlock) void mx_join_kernel(MxMatmulArgs a, uint32_t splits) {
  using TO = typename Num<DO>::T;
  const uint64_t n = a.M * a.N;
  for (uint64_t e = ((uint64_t)blockIdx.x * kBlock + threadIdx.x) * 4; e < n; e += (uint64_t)gridDim.x * kBlock * 4) {
    v4f s{0, 0, 0, 0};
    for (uint32_t k = 0; k < splits; ++k) s += load4(a.ws + k * n, e, n);
    store4<TO>(static_cast<TO *>(a.y), e, n, s);
  }
}

// Which kernel, and how often k is cut.
struct Plan {
  enum { kDirect, kMiddle, kBig } kind;
  uint32_t tiles_m, tiles_n, splits, stages_each;
};

Plan plan_of(uint64_t M, uint64_t N, uint32_t K) {
  Plan p{Plan::kDirect, 0, 0, 1, 1};
  // Few rows, or so few outputs that one round of the direct kernel's workgroups covers
  // them (8192 x 8192 weights: 16 rows of e2m1 11.5 us against 15.2 for the tiles, 32 rows 20.1
  // against 15.3; of e4m3 15.8 against 25.9, 28.2 against 25.6).
  const uint64_t blocks = ((M + 15) / 16) * ((N + 15) / 16);
  if (blocks <= 512 || (M <= 16 && blocks <= 1u << 22)) return p;
  // Many rows: the larger tiles from 192 of them on (e2m1: 1536 x 8192 outputs, 4096 deep 34
  // us against 45, 8192 deep 60 against 83; 1024 x 8192, 8192 deep, 128 large tiles: 54 each;
  // e4m3: 82 against 97, 137 against 183; 136 against 108).
  const bool big = ((M + 255) / 256) * ((N + 255) / 256) >= 192;
  const uint32_t wide = big ? 256 : 128;
  p.kind = big ? Plan::kBig : Plan::kMiddle;
  p.tiles_m = (uint32_t)((M + wide - 1) / wide);
  p.tiles_n = (uint32_t)((N + wide - 1) / wide);
  const uint64_t tiles = (uint64_t)p.tiles_m * p.tiles_n;
  const uint32_t stages = (uint32_t)((mx_blocks(K) + 3) / 4);
  // One workgroup takes half a microsecond a stage however few there are: k is cut into
  // ranges of whole scale groups (4 stages), at least 8 stages each, until there is one per
  // CU (128 x 8192 outputs, 8192 deep: e2m1 31 us in one range, 19.3 in four; e4m3 73, 29.7),
  // eight at most, for as much workspace each as 32-bit results take (384 x 384 outputs, 8192
  // deep, e2m1: 13.4 in eight, 16.4 in sixteen; 256 x 1024, 65536 deep: 38, 29).
  const uint64_t want = big ? 1 : 256 / tiles, most = stages / 8;
  uint32_t n = (uint32_t)(want < most ? want : most);
  n = n < 1 ? 1 : (n > 8 ? 8 : n);
  p.stages_each = ((stages + n - 1) / n + 3) / 4 * 4;
  if (p.stages_each == 0) p.stages_each = 4;
  p.splits = stages ? (stages + p.stages_each - 1) / p.stages_each : 1;
  return p;
}

// The large tile's wavefronts and fragments: few fragments of e4m3 a wavefront, as it splits each.
struct BigTile { int wm, wn, fm, fn; };
template <bool A8> constexpr BigTile kBigTile = A8 ? BigTile{4, 2, 4, 8} : BigTile{2, 4, 8, 4};

template <bool A8, int DO> hipError_t go_tile(const MxMatmulArgs &a, const Plan &p, void *dst, hipStream_t s) {
  const dim3 grid(p.tiles_m * p.tiles_n, p.splits);
  if (p.kind == Plan::kBig)
    mx_tile_kernel<false, A8, kBigTile<A8>.wm, kBigTile<A8>.wn, kBigTile<A8>.fm, kBigTile<A8>.fn, DO><<<grid, 512, 0, s>>>(a, dst, p.tiles_m, p.tiles_n, p.stages_each);
  else
    mx_tile_kernel<false, A8, 2, 2, 4, 4, DO><<<grid, 256, 0, s>>>(a, dst, p.tiles_m, p.tiles_n, p.stages_each);
  return hipGetLastError();
}

template <bool A8> hipError_t go(const MxMatmulArgs &a, hipStream_t s) {
  const Plan p = plan_of(a.M, a.N, a.K);
  if (p.kind == Plan::kDirect) return go_direct<A8>(a, s);
  if ((uint64_t)p.tiles_m * p.tiles_n > 0x7FFFFF) return hipErrorInvalidValue;
  if (p.splits > 1) {
    const hipError_t e = go_tile<A8, IBP_F32>(a, p, a.ws, s);
    if (e != hipSuccess) return e;
  }
  return with_dtype(a.dtype, [&](auto d) {
    if (p.splits == 1) return go_tile<A8, d.value>(a, p, a.y, s);
    const uint64_t n = (a.M * a.N + kBlock * 4 - 1) / (kBlock * 4);
    mx_join_kernel<d.value><<<(uint32_t)(n < 4096 ? n : 4096), kBlock, 0, s>>>(a, p.splits);
    return hipGetLastError();
  });
}

// ------------------------------------------------------------------ rows of experts

// A few rows an expert: bound by reading the weights.  A workgroup of four wavefronts
// computes 16 FM rows of one expert by 64 FN columns, each wavefront all rows of 16 FN columns.
// Operands come as in the larger tiles, in a ring of three stages of 128 elements; one barrier a
// stage, at which its loads are done and all have read the stage before, whose place is
// filled anew.  Three workgroups a CU overlap their loads and products (with five stages two
// fit: 64 rows of 64 experts, 2048 x 4096, e4m3 36.2 us against 33.4, 4.4 TB/s of weights; 1501 of
// 24, 1000 x 1503, one or two workgroups a CU, e2m1 9.3 and 9.1, e4m3 15.4 and 14.6).  Of 64 rows
// of e4m3 all four wavefronts split the same codes, ten vector instructions to a matrix one (2048
// rows of 32 ragged experts, 2048 x 4096: 62 us, e2m1, which has nothing to split, 39).
template <bool A8, int FM, int FN, int DO>
__global__ __launch_bounds__(256) void mx_rows_kernel(MxMatmulArgs a, uint32_t tiles_n) {
  using TO = typename Num<DO>::T;
  constexpr uint32_t kWaves = 4, kStages = 3, kPitchA = A8 ? 128 : 64, kPitchB = 64, kRowsB = 64 * FN;
  constexpr uint32_t kLeastA = 1024 * kWaves / kPitchA;  // rows that a load of every wavefront covers
  constexpr uint32_t kRowsA = 16 * FM < kLeastA ? kLeastA : 16 * FM;
  using TileA = Tile<kRowsA, kPitchA, kWaves>;
  using TileB = Tile<kRowsB, kPitchB, kWaves>;
  constexpr uint32_t kStage = TileA::kBytes + TileB::kBytes, kLoads = TileA::kLoads + TileB::kLoads;
  // scales of four stages, 16 bytes of each row of A, then of B
  constexpr uint32_t kGroup = 4, kLoaders = (16 * FM + kRowsB + 63) / 64, kScales = kLoaders * 1024;
  static_assert(kStages - 1 <= kGroup, "a stage is asked for after its scales");
  static_assert(kLoaders <= kWaves && (kStages - 2) * kLoads < 64, "");
  __shared__ __align__(1024) uint8_t ring[kStages * kStage + 2 * kScales];
  const uint32_t lane = lane_id(), wave = uniform(threadIdx.x / kWave), r = lane & 15, g = lane >> 4;
  const Experts x{a.offsets, a.experts, (uint32_t)__builtin_ctz(16 * FM), a.M};
  const uint32_t block = blockIdx.y * gridDim.x + blockIdx.x;
  if (a.err && block == 0 && wave == 0) check_offsets(x, a.err);
  const UnitSearch<false> search(x);
  if (block >= (uint64_t)search.total * tiles_n) return;
  const TileId t = tile_of(block, search.total, tiles_n);
  const Unit u = search.find(t.row);
  if (u.row0 >= u.end) return;
  const uint64_t m0 = u.row0, n0 = (uint64_t)t.col * kRowsB;
  a.b_codes += u.expert * a.N * mx_code_pitch(a.K, false);
  a.b_scales += u.expert * a.N * mx_scale_pitch(a.K);
  const uint32_t nblk = (uint32_t)mx_blocks(a.K), sp = (uint32_t)mx_scale_pitch(a.K);
  const uint32_t cpa = (uint32_t)mx_code_pitch(a.K, A8), cpb = (uint32_t)mx_code_pitch(a.K, false);
  TileA ta;
  TileB tb;
  ta.init(a.a_codes, m0, u.end, cpa, wave, lane);
  tb.init(a.b_codes, n0, a.N, cpb, wave, lane);
  const uint8_t *scale;
  {
    const uint32_t row = wave * 64 + lane;
    const bool of_a = row < 16 * FM;
    const uint64_t at = of_a ? m0 + row : n0 + row - 16 * FM, rows = of_a ? u.end : a.N;
    scale = (of_a ? a.a_scales : a.b_scales) + (at < rows ? at : rows - 1) * sp;
  }
  v4f acc[FN][FM];
#pragma unroll
  for (int n = 0; n < FN; ++n)
#pragma unroll
    for (int m = 0; m < FM; ++m) acc[n][m] = v4f{0, 0, 0, 0};
  uint8_t *const scales = ring + kStages * kStage;
  // Always kLoads loads, of zeros past the rows' end: the waits below count on it.
  auto fill = [&](uint8_t *st, uint32_t stage) {
    ta.load(st, stage * kPitchA, cpa, wave);
    tb.load(st + TileA::kBytes, stage * kPitchB, cpb, wave);
  };
  // as in the larger tiles
  auto fill_scales = [&](uint8_t *sc, uint32_t q) {
    if (wave >= kLoaders) return;
    if ((q + 1) * 16 <= sp) {
      to_lds16(scale + q * 16, sc + wave * 1024);
    } else {
      uint32_t d[kGroup];
#pragma unroll
      for (uint32_t j = 0; j < kGroup; ++j)
        d[j] = q * 16 + j * 4 < sp ? *reinterpret_cast<const uint32_t *>(scale + q * 16 + j * 4) : 0u;
      *reinterpret_cast<uint4 *>(sc + wave * 1024 + lane * 16) = make_uint4(d[0], d[1], d[2], d[3]);
    }
  };
  const uint32_t steps = (nblk + 3) / 4, wn = wave * 16 * FN;
  const uint32_t at_a = r * kPitchA + swizzle<kPitchA>(r, g) * 16, at_a2 = r * kPitchA + swizzle<kPitchA>(r, 4 + g) * 16;
  const uint32_t at_b = TileA::kBytes + (wn + r) * kPitchB + swizzle<kPitchB>(r, g) * 16;
  v8i w[FN], v[FM];
  int ws[FN], xs[FM];
  // What is filled is not what is read; __restrict__ says so to the compiler, which
  // otherwise would wait for all loads in flight before an LDS read.
  auto read = [&](uint8_t *__restrict__ filled, uint8_t *__restrict__ filled_scales, const uint8_t *__restrict__ st,
                  const uint8_t *__restrict__ sc, uint32_t k) {
    if (k % kGroup == 0) fill_scales(filled_scales, k / kGroup + 1);
    fill(filled, k + kStages - 1);
    const uint4 none = make_uint4(0u, 0u, 0u, 0u);
#pragma unroll
    for (int n = 0; n < FN; ++n) {
      w[n] = operand(*reinterpret_cast<const uint4 *>(st + at_b + n * 16 * kPitchB), none);
      ws[n] = sc[(16 * FM + wn + r) * 16 + g + n * 256];
    }
#pragma unroll
    for (int m = 0; m < FM; ++m) {
      v[m] = operand(*reinterpret_cast<const uint4 *>(st + at_a + m * 16 * kPitchA),
                     A8 ? *reinterpret_cast<const uint4 *>(st + at_a2 + m * 16 * kPitchA) : none);
      xs[m] = sc[r * 16 + g + m * 256];
    }
  };
  fill_scales(scales, 0);
#pragma unroll
  for (uint32_t k = 0; k + 1 < kStages; ++k) fill(ring + k * kStage, k);
  uint32_t now = 0, next = kStages - 1;
#pragma unroll 1
  for (uint32_t k = 0; k < steps; ++k) {
    __builtin_amdgcn_s_waitcnt(wait_loads_and_lds((kStages - 2) * kLoads));
    phase_barrier();
    const uint32_t odd = k / kGroup & 1;
    read(ring + next * kStage, scales + (odd ^ 1) * kScales, ring + now * kStage, scales + odd * kScales + k % kGroup * 4, k);
    next = now;
    now = now + 1 == kStages ? 0 : now + 1;
#pragma unroll
    for (int m = 0; m < FM; ++m)
#pragma unroll
      for (int n = 0; n < FN; ++n) acc[n][m] = mfma_mx<A8>(w[n], v[m], acc[n][m], ws[n], xs[m]);
  }
  __builtin_amdgcn_s_waitcnt(kWaitVmcnt0);  // no load into LDS outlives the workgroup
  TO *y = static_cast<TO *>(a.y);
#pragma unroll
  for (int m = 0; m < FM; ++m) {
    const uint64_t gm = m0 + 16 * m + r;
    if (gm >= u.end) continue;
#pragma unroll
    for (int n = 0; n < FN; ++n) store4<TO>(y + gm * a.N, n0 + wn + 16 * n + 4 * g, a.N, acc[n][m]);
  }
}

template <bool A8, int FM> hipError_t go_rows(const MxMatmulArgs &a, hipStream_t s) {
  constexpr uint32_t kCols = 128;
  const uint64_t tiles_n = (a.N + kCols - 1) / kCols;
  const uint64_t grid = most_units(a.M, a.experts, __builtin_ctz(16 * FM), false) * tiles_n;
  const uint64_t many = (grid + (1u << 20) - 1) >> 20;  // a dimension of a launch holds less than 2^24 workgroups of 256
  return with_dtype(a.dtype, [&](auto d) {
    mx_rows_kernel<A8, FM, kCols / 64, d.value><<<dim3((uint32_t)(many > 1 ? 1u << 20 : grid), (uint32_t)many), 256, 0, s>>>(a, (uint32_t)tiles_n);
    return hipGetLastError();
  });
}

template <bool A8> hipError_t go_grouped(const MxMatmulArgs &a, hipStream_t s) {
  const uint64_t T = a.M, E = a.experts, units = most_units(T, E, 4, false);
  // So little work that the direct kernel's wavefronts, which share k, are not many either (2
  // rows of 8 experts, 4096 x 4096, e4m3 7.0 us against 14.5; 90 of 3, 2000 x 2000 6.1 and 9.1;
  // 8 of 64, 2048 x 4096 11.1 and 15.3; 16 of 64 21.5 and 16.6; 300 of 8, 1000 x 1000 8.1 and 6.6).
  if (units * ((a.N + 63) / 64) <= 256) {
    const uint32_t steps = (uint32_t)((mx_blocks(a.K) + kStep - 1) / kStep);
    uint32_t waves = 4;
    while (waves > 1 && waves > steps) waves /= 2;
    return with_dtype(a.dtype, [&](auto d) {
      mx_direct_kernel<true, A8, d.value><<<dim3((uint32_t)((a.N + 15) / 16), (uint32_t)units), waves * kWave, (waves - 1) * 1024, s>>>(a);
      return hipGetLastError();
    });
  }
  // The rest goes by the rows an expert has on average, as their number is all that the host
  // knows, and by the tiles that they make, half a tile more an expert.  256 x 256 tiles (32
  // experts, 2048 x 4096, ragged, e4m3): 8192 rows 149 us, with 128 x 128 tiles 152, evenly
  // spread 86 and 109; 4096 rows 146 and 101; 4096 rows of 4 experts, 4096 x 4096 (288 tiles) 147
  // and 143.  128 x 128: 4096 rows 101, with 64 rows by 128 columns 108, of e2m1 49 and 59; 2048
  // rows 90 and 62, 45 and 40; 800 rows of 4 experts, 4096 x 2048 (256 tiles) 24.0 and 24.0, 2000
  // of 8, 500 x 500 (80 tiles) 10.4 and 7.7.
  auto tiles = [&](uint64_t wide) { return (T / wide + E / 2) * ((a.N + wide - 1) / wide); };
  const bool big = T >= 192 * E && tiles(256) >= 384, middle = T >= 112 * E && tiles(128) >= 256;
  if (big || middle) {
    const uint32_t wide = big ? 256 : 128, each = (uint32_t)((mx_blocks(a.K) + 15) / 16 * 4);
    const uint64_t tiles_n = (a.N + wide - 1) / wide, grid = most_units(T, E, big ? 8 : 7, false) * tiles_n;
    if (grid > 0x7FFFFF) return hipErrorInvalidValue;
    return with_dtype(a.dtype, [&](auto d) {
      if (big) mx_tile_kernel<true, A8, kBigTile<A8>.wm, kBigTile<A8>.wn, kBigTile<A8>.fm, kBigTile<A8>.fn, d.value><<<(uint32_t)grid, 512, 0, s>>>(a, a.y, 0, (uint32_t)tiles_n, each);
      else mx_tile_kernel<true, A8, 2, 2, 4, 4, d.value><<<(uint32_t)grid, 256, 0, s>>>(a, a.y, 0, (uint32_t)tiles_n, each);
      return hipGetLastError();
    });
  }
  // Fewer rows a tile read and split fewer codes for nothing, more read the weights less often
  // (32 ragged experts, 2048 x 4096; tiles of 16, 32 and 64 rows; e4m3: 512 rows 33, 38, 42 us,
  // 1024 rows 50, 39, 59, 2048 rows 75, 63, 62; e2m1: 512 rows 31.6, 34.3, 29.0, 2048 rows 72, 52,
  // 39; 256 rows of 128 experts, 768 x 2048 16.8, 16.9, 17.5).
  if constexpr (A8) {
    if (T <= 16 * E) return go_rows<true, 1>(a, s);
    return T <= 48 * E ? go_rows<true, 2>(a, s) : go_rows<true, 4>(a, s);
  } else {
    return T < 8 * E ? go_rows<false, 2>(a, s) : go_rows<false, 4>(a, s);
  }
}

}  // namespace

hipError_t launch_mx_grouped_matmul(const MxMatmulArgs &a, hipStream_t s) {
  return a.a_e4m3 ? go_grouped<true>(a, s) : go_grouped<false>(a, s);
}

uint64_t mx_matmul_workspace(uint64_t M, uint64_t N, uint32_t K) {
  const Plan p = plan_of(M, N, K);
  return p.splits > 1 ? p.splits * M * N * 4 : 0;
}

hipError_t launch_mx_matmul(const MxMatmulArgs &a, hipStream_t s) {
  return a.a_e4m3 ? go<true>(a, s) : go<false>(a, s);
}

}  // namespace ibp
