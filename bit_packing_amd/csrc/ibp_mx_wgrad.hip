// ibp_mx_wgrad.hip -- weight gradient of a linear layer from the 8-bit checkpoint of its
// input: dW[o][i] = sum over tokens t of dY[t][o] X[t][i], X packed as e4m3.
//
// An e4m3 value times its power-of-two scale (at least 2^-117) is a BF16 number, so X is
// decoded exactly to BF16 and the product runs on the BF16 matrix instruction with 32-bit
// sums.  A dY of another type is the sum of BF16 numbers, two for half precision's 11 bits
// and three for single's 24, each the leading eight bits of what the ones before leave; each
// part has its own ranges of the launch and is added like another range.  Both operands lie
// with t as the slow dimension, while the instruction wants consecutive t in a lane: tiles
// are staged in LDS as they lie and read through the transposing LDS read, which hands each
// of 16 lanes one column of a 4 x 16 block.
#include "ibp_device.h"
#include "ibp_num.h"
#include "ibp_tile.h"

namespace ibp {
namespace {

using namespace dev;

typedef short v4s __attribute__((ext_vector_type(4)));
typedef uint32_t v2u __attribute__((ext_vector_type(2)));
typedef __bf16 v8b __attribute__((ext_vector_type(8)));
typedef float v16f __attribute__((ext_vector_type(16)));

constexpr uint32_t kT = 32;  // tokens per stage

// The 32-byte pieces of row t of a tile are permuted by three bits of t, so that what half a
// wavefront reads at a time falls into all 64 banks: for fragments of F = 16 columns a piece
// of each of eight rows, for F = 32 two neighbouring pieces of each of four.
template <int F> __device__ __forceinline__ uint32_t permute(uint32_t piece, uint32_t t) {
  return piece ^ (F == 16 ? t & 7 : (t & 3) << 1 | (t >> 2 & 1));
}

// LDS byte of the 16-byte piece `c16` of row t of a tile of W columns.
template <uint32_t W, int F> __device__ __forceinline__ uint32_t tile_at(uint32_t t, uint32_t c16) {
  return t * (W * 2) + (permute<F>(c16 >> 1, t) << 5 | (c16 & 1) << 4);
}

// Eight BF16 of column block `col` (F columns) of a stage's tokens from 16 s on, in the order
// of the matrix instruction's k: lane group g of F lanes takes rows 4 g .. 4 g + 3 and as many
// 16 (F = 16) or 8 rows further on; both operands do, so the sum is over the same tokens.
template <uint32_t W, int F> __device__ __forceinline__ v8b fragment(const uint8_t *tile, uint32_t col, uint32_t s, uint32_t lane) {
  const uint32_t t = lane / F * 4 + ((lane & 15) >> 2), piece = F == 16 ? col : col * 2 + (lane >> 4 & 1);
  const uint8_t *at = tile + (16 * s + t) * (W * 2) + (permute<F>(piece, t) << 5) + (lane & 3) * 8;
  using L = __attribute__((address_space(3))) v4s;
  const v4s lo = __builtin_amdgcn_ds_read_tr16_b64_v4i16((L *)at);
  const v4s hi = __builtin_amdgcn_ds_read_tr16_b64_v4i16((L *)(at + (F == 16 ? 16 : 8) * W * 2));
  return __builtin_bit_cast(v8b, __builtin_shufflevector(lo, hi, 0, 1, 2, 3, 4, 5, 6, 7));
}

// Eight e4m3 codes of one block as BF16, exactly.
__device__ __forceinline__ v8b decode8(v2u q, float f) {
  typedef __bf16 v2b __attribute__((ext_vector_type(2)));
  const v2b a = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(q.x, f, false);
  const v2b b = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(q.x, f, true);
  const v2b c = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(q.y, f, false);
  const v2b d = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(q.y, f, true);
  return v8b{a[0], a[1], b[0], b[1], c[0], c[1], d[0], d[1]};
}

// Part `part` of eight elements as BF16: the leading eight bits of what the parts before
// leave.  Cutting, not rounding, leaves the largest finite values finite, and the last
// part holds all that is left.  Infinities and NaNs are in the first part alone.
template <typename TY> __device__ __forceinline__ v8b part_of(Vec8<TY> y, uint32_t part) {
  if constexpr (std::is_same<TY, __bf16>::value) {
    return (v8b)y;
  } else {
    v8b out;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      float rest = (float)y[i];
      const bool finite = (__builtin_bit_cast(uint32_t, rest) & 0x7F800000u) != 0x7F800000u;
      for (uint32_t p = 0; p < part; ++p) rest -= __builtin_bit_cast(float, __builtin_bit_cast(uint32_t, rest) & 0xFFFF0000u);
      // a NaN's payload may lie in the bits that are cut off
      const float cut = __builtin_bit_cast(float, __builtin_bit_cast(uint32_t, rest) & 0xFFFF0000u);
      out[i] = (__bf16)(finite ? cut : (part == 0 ? rest : 0.0f));
    }
    return out;
  }
}

// A load that the compiler knows to be of global memory: from a pointer chosen between a
// matrix and kZeros it would make a flat load, which LDS waits count too.
template <typename T> __device__ __forceinline__ T from_global(const uint8_t *p) {
  return *reinterpret_cast<const __attribute__((address_space(1))) T *>((uintptr_t)p);
}

// A workgroup of WI x WO wavefronts computes F FI WI (i) by F FO WO (o) elements of dW
// over the tokens [z * t_each, (z + 1) * t_each), z = blockIdx.y % splits, of part
// blockIdx.y / splits of dY, into dst + blockIdx.y * N * K.
//
// Stages of 32 tokens lie in a ring of four.  dY comes by direct global-to-LDS loads three
// stages ahead where its rows are aligned to 16 bytes (DIRECT: they are, or wgrad_parts_kernel
// has laid them out so; part p is then T rows further on), else through registers like
// X, which is loaded four stages ahead and decoded into LDS two stages ahead.  As in the
// 4-bit product, half of the eight wavefronts of a large tile read a stage while the other
// half multiplies (16384 x 4096 x 8192: 859 us, 1.28 PFLOP/s, against 1090 with all in
// step and two stages of 64 tokens).  Bound by the phases (the matrix units are busy 57% of the
// time, LDS 28%) and by power: the clock falls to 1.9 to 2.1 GHz.
//
// F = 32 takes the 32 x 32 x 16 matrix instruction: a third more from registers alone, at more
// power.  The large tile is 11% slower in clock for 8% fewer cycles with it (894 us against
// 862) and takes F = 16; the small one, bound by latency, is faster (999 x 504 x 1000 14.5 us
// against 15.3, 16384 x 256 x 256 23.5 against 25.5).
template <int F, int WI, int WO, int FI, int FO, bool DIRECT, int DY, int DO>
__global__ __launch_bounds__(WI *WO *64) void wgrad_kernel(MxWgradArgs a, void *dst, uint64_t t_each, uint32_t tiles_o,
                                                           uint32_t tiles_i, uint32_t splits) {
  using TY = typename Num<DY>::T;
  static_assert(!DIRECT || DY == IBP_BF16, "");
  using TO = typename Num<DO>::T;
  constexpr uint32_t kWaves = WI * WO, kThreads = kWaves * 64, kWideI = F * FI * WI, kWideO = F * FO * WO;
  constexpr uint32_t kPiecesY = kT * kWideO / 8 / kThreads, kPiecesX = kT * kWideI / 8 / kThreads;
  constexpr uint32_t kBytesY = kT * kWideO * 2, kStage = kBytesY + kT * kWideI * 2, kRing = 4;
  constexpr uint32_t kStepY = kThreads / (kWideO / 8), kStepX = kThreads / (kWideI / 8);  // tokens between a thread's pieces
  static_assert(kStepY % 8 == 0 && kStepX % 8 == 0, "the permutation goes by t & 7, the same for all pieces of a thread");
  __shared__ __align__(1024) uint8_t ring[kRing * kStage];
  const uint32_t lane = lane_id(), wave = uniform(threadIdx.x / kWave);
  const TileId tile = tile_of(blockIdx.x, tiles_o, tiles_i);
  const uint32_t o0 = tile.row * kWideO, i0 = tile.col * kWideI;
  const uint32_t wi = (wave % WI) * FI, wo = (wave / WI) * FO;  // in blocks of F
  const uint32_t part = blockIdx.y / splits;
  const uint64_t t0 = (blockIdx.y - part * splits) * t_each, t1 = t0 + t_each < a.T ? t0 + t_each : a.T;
  const uint32_t cp = (uint32_t)mx_code_pitch(a.K, true), sp = (uint32_t)mx_scale_pitch(a.K);
  const TY *dy = static_cast<const TY *>(a.dy);

  // A thread's pieces lie at one column, so a pointer each for dY, codes and scales walks
  // over the tokens; past a row's end it stands still on zeros.
  const uint32_t ty = threadIdx.x / (kWideO / 8), sy = threadIdx.x % (kWideO / 8);
  const uint32_t tx = threadIdx.x / (kWideI / 8), sx = threadIdx.x % (kWideI / 8), cx = i0 + sx * 8;
  // LDS takes dY's pieces in lane order; the permutation is made by their sources
  const uint32_t cy = o0 + (permute<F>(sy >> 1, ty) << 1 | (sy & 1)) * 8;
  const bool in_y = !DIRECT || cy < a.dy_pitch, in_x = cx < cp;
  // without DIRECT a piece past the row's end is the row's last eight elements (load8)
  const bool wide = a.N >= 8;
  const uint64_t at_y = DIRECT ? cy : (wide ? (cy + 8 <= a.N ? cy : a.N - 8) : 0);
  const uint64_t row_y = t0 + ty + (DIRECT ? part * a.T : 0);
  const uint8_t *py = in_y ? reinterpret_cast<const uint8_t *>(dy + row_y * a.dy_pitch + at_y) : kZeros;
  const uint8_t *px = in_x ? a.x_codes + (t0 + tx) * cp + cx : kZeros;
  const uint8_t *ps = in_x ? a.x_scales + (t0 + tx) * sp + cx / (4 * kMxBlock) * 4 : kZeros;  // its dword
  const uint32_t scale_shift = cx / kMxBlock % 4 * 8;
  const uint64_t go_y = in_y ? (uint64_t)kStepY * a.dy_pitch * sizeof(TY) : 0, go_x = in_x ? (uint64_t)kStepX * cp : 0;
  const uint64_t go_s = in_x ? (uint64_t)kStepX * sp : 0;
  const uint32_t at_x = kBytesY + tile_at<kWideI, F>(tx, sx);

  using Acc = typename std::conditional<F == 16, v4f, v16f>::type;
  Acc acc[FI][FO];
#pragma unroll
  for (int x = 0; x < FI; ++x)
#pragma unroll
    for (int y = 0; y < FO; ++y) acc[x][y] = Acc{};

  // An even number of stages, the last perhaps of zeros: the loop takes two at a time, so
  // that the two sets of registers of loads in flight are known to the compiler.
  const uint32_t steps = t0 < t1 ? (uint32_t)((t1 - t0 + 2 * kT - 1) / (2 * kT)) * 2 : 0;
  const uint32_t tokens = t0 < t1 ? (uint32_t)(t1 - t0) : 0;
  struct Set {
    v2u q[kPiecesX];
    uint32_t s[kPiecesX];
    Vec8<TY> y[DIRECT ? 1 : kPiecesY];
  } set[2];
  // Loads of a stage; stages are asked for in order.  Their number never varies (zeros
  // past the last token), as the waits below count them.
  auto fetch = [&](Set &f, uint32_t stage) {
#pragma unroll
    for (uint32_t p = 0; p < kPiecesX; ++p) {
      const bool in = stage * kT + tx + p * kStepX < tokens;
      f.q[p] = from_global<v2u>(in ? px : kZeros);
      f.s[p] = from_global<uint32_t>(in ? ps : kZeros);
      px += go_x;
      ps += go_s;
    }
    if constexpr (!DIRECT) {
#pragma unroll
      for (uint32_t p = 0; p < kPiecesY; ++p) {
        const uint8_t *from = stage * kT + ty + p * kStepY < tokens ? py : kZeros;
        f.y[p] = wide ? from_global<Vec8<TY>>(from) : load8<false, TY>(reinterpret_cast<const TY *>(from), 0, a.N);
        py += go_y;
      }
    }
  };
  auto fetch_direct = [&](uint8_t *st, uint32_t stage) {
    if constexpr (DIRECT) {
#pragma unroll
      for (uint32_t p = 0; p < kPiecesY; ++p) {
        to_lds16(stage * kT + ty + p * kStepY < tokens ? py : kZeros, st + (p * kWaves + wave) * 1024);
        py += go_y;
      }
    }
  };
  // what came through registers goes to LDS
  auto settle = [&](uint8_t *st, const Set &f) {
    if constexpr (!DIRECT) {
#pragma unroll
      for (uint32_t p = 0; p < kPiecesY; ++p)
        *reinterpret_cast<v8b *>(st + (p * kThreads + threadIdx.x) * 16) =
            part_of<TY>(wide ? settle8<true, TY>(f.y[p], cy, a.N) : settle8<false, TY>(f.y[p], cy, a.N), part);
    }
#pragma unroll
    for (uint32_t p = 0; p < kPiecesX; ++p)
      *reinterpret_cast<v8b *>(st + at_x + p * kStepX * kWideI * 2) = decode8(f.q[p], mx_factor((f.s[p] >> scale_shift) & 0xFFu));
  };
  auto barrier = [&] {
    asm volatile("" ::: "memory");
    __builtin_amdgcn_sched_barrier(0);
    __builtin_amdgcn_s_barrier();
    __builtin_amdgcn_sched_barrier(0);
    asm volatile("" ::: "memory");
  };
  // A turn is a reading phase and a multiplying phase with a barrier after each; with two
  // wavefronts a SIMD the second half of them runs one phase behind the first.
  constexpr bool kPingPong = kWaves == 8;
  const bool behind = kPingPong && wave >= kWaves / 2;
  constexpr uint32_t kLoads = 2 * kPiecesX + kPiecesY;  // a wavefront's per turn
  static_assert(kLoads < 16, "");
  constexpr uint32_t kDeep = F == 16 ? 1 : 2;  // matrix instructions that a stage is deep
  v8b fx[kDeep][FI], fy[kDeep][FO];
  // What the loads in flight fill is not what is read; __restrict__ says so to the compiler,
  // which otherwise would wait for all of them before an LDS read.
  auto read = [&](uint8_t *__restrict__ filled, const uint8_t *__restrict__ now) {
    (void)filled;
#pragma unroll
    for (uint32_t s = 0; s < kDeep; ++s) {
#pragma unroll
      for (int y = 0; y < FO; ++y) fy[s][y] = fragment<kWideO, F>(now, wo + y, s, lane);
#pragma unroll
      for (int x = 0; x < FI; ++x) fx[s][x] = fragment<kWideI, F>(now + kBytesY, wi + x, s, lane);
    }
  };
  auto write = [&](uint8_t *__restrict__ filled, uint8_t *__restrict__ settled, Set &f, uint32_t k) {
    settle(settled, f);
    fetch(f, k + 4);
    fetch_direct(filled, k + 3);
  };
  auto turn = [&](Set &f, uint32_t k) {
    read(ring + ((k + 3) % kRing) * kStage, ring + (k % kRing) * kStage);
    // These reads are done, and this wavefront's direct loads of stage k + 1 (of turn k - 2;
    // turn k - 1's are not waited for): after two barriers the first half reads it.
    __builtin_amdgcn_s_waitcnt(0xC07F);
    if constexpr (DIRECT) __builtin_amdgcn_s_waitcnt(0x0F70 | kLoads);
    barrier();
    __builtin_amdgcn_s_setprio(1);
#pragma unroll
    for (uint32_t s = 0; s < kDeep; ++s) {
#pragma unroll
      for (int x = 0; x < FI; ++x) {
#pragma unroll
        for (int y = 0; y < FO; ++y) {
          if constexpr (F == 16) acc[x][y] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(fx[s][x], fy[s][y], acc[x][y], 0, 0, 0);
          else acc[x][y] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(fx[s][x], fy[s][y], acc[x][y], 0, 0, 0);
        }
        if (s == 0 && x == 0) {
          __builtin_amdgcn_sched_barrier(0);  // the compiler would put this before the matrix instructions
          write(ring + ((k + 3) % kRing) * kStage, ring + ((k + 2) % kRing) * kStage, f, k);
        }
      }
    }
    __builtin_amdgcn_sched_barrier(0);
    __builtin_amdgcn_s_setprio(0);
    barrier();
  };
  if (steps) {
#pragma unroll
    for (uint32_t k = 0; k < 3; ++k) fetch_direct(ring + k * kStage, k);
#pragma unroll
    for (uint32_t k = 0; k < 2; ++k) fetch(set[k], k);
#pragma unroll
    for (uint32_t k = 0; k < 2; ++k) settle(ring + k * kStage, set[k]);
#pragma unroll
    for (uint32_t k = 0; k < 2; ++k) fetch(set[k], k + 2);
    __builtin_amdgcn_s_waitcnt(kWaitVmcnt0 & ~0x0F00);  // and LDS writes
  }
  barrier();
  if (behind) barrier();
#pragma unroll 1
  for (uint32_t k = 0; k < steps; k += 2) {
    turn(set[0], k);
    turn(set[1], k + 1);
  }
  if (kPingPong && !behind) barrier();
  __builtin_amdgcn_s_waitcnt(kWaitVmcnt0);  // no load into LDS outlives the workgroup
  // a lane has once or four times four consecutive i of one o
  TO *dw = static_cast<TO *>(dst) + (uint64_t)blockIdx.y * a.N * a.K;
#pragma unroll
  for (int y = 0; y < FO; ++y) {
    const uint32_t o = o0 + (wo + y) * F + lane % F;
    if (o >= a.N) continue;
#pragma unroll
    for (int x = 0; x < FI; ++x) {
#pragma unroll
      for (int q = 0; q < F * F / 256; ++q)
        store4<TO>(dw + (uint64_t)o * a.K, i0 + (wi + x) * F + 8 * q + 4 * (lane / F), a.K,
                   v4f{acc[x][y][4 * q], acc[x][y][4 * q + 1], acc[x][y][4 * q + 2], acc[x][y][4 * q + 3]});
    }
  }
}

// Lays dY out as the large tile's direct loads want it: its parts in BF16, T rows each, rows
// filled up with zeros to a multiple of eight elements.  One pass; 16001 tokens of 1153, 4097
// inputs: 198 us with it, against 300 through registers; 8192 x 4096 x 4096 in single
// precision 778 against 2027, 4096 x 2048 x 2048 in half precision 105 against 188.  The small
// tile takes such a dY through registers, without a launch more (999 x 500 x 1000 18.6 us,
// 14.6 with 504).
template <int DY> __global__ __launch_bounds__(kBlock) void wgrad_parts_kernel(MxWgradArgs a, __bf16 *out, uint32_t parts) {
  using TY = typename Num<DY>::T;
  const TY *dy = static_cast<const TY *>(a.dy);
  const uint32_t pieces = a.dy_pitch / 8;
  const uint64_t n = a.T * pieces, step = (uint64_t)gridDim.x * kBlock;
  by_width(a.N, [&](auto wide) {
    for (uint64_t e = (uint64_t)blockIdx.x * kBlock + threadIdx.x; e < n; e += step) {
      const uint64_t t = e / pieces;
      const uint32_t c = (uint32_t)(e - t * pieces) * 8;
      const Vec8<TY> y = settle8<wide.value, TY>(load8<wide.value, TY>(dy + t * a.N, c, a.N), c, a.N);
      for (uint32_t p = 0; p < parts; ++p) *reinterpret_cast<v8b *>(out + ((p * a.T + t) * pieces * 8 + c)) = part_of<TY>(y, p);
    }
  });
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

// Tile and ranges of tokens.  256 x 256 tiles read each operand half as often as 128 x 128
// ones, but half as many fit: two small workgroups share a CU.  The large ones are taken where
// the small ones would not fit at once (256 large tiles: 128 tokens 23 us against 25, 500 32
// against 38; 160: 1000 tokens 37 against 43), and where the tokens make up for the CUs left
// empty (128: 2000 tokens 55 against 47, 4000 81 against 83, 8000 132 against 154; 16: 8000
// 42 against 41, 16000 56 against 66; 4: 16000 38 against 29).
// The tokens are cut into ranges until there is a workgroup per CU (16384 tokens of 1024 x
// 1024: 366 us in one range, 55 in sixteen), each of 256 tokens at least, 32 ranges at most: a
// range's sums are written and read once in 32 bits (256 x 256: 16384 tokens 22.5 us in 32
// ranges, 29.6 in 64, 65536 tokens 39.9 and 39.2; 128 x 128, 262144 tokens 198 and 116).
struct Plan {
  bool big;
  bool copied;  // dY laid out anew, as the large tile takes it
  uint32_t tiles_o, tiles_i;
  uint32_t splits;
  uint32_t parts;  // of dY
  uint64_t t_each;

  uint64_t pieces() const { return (uint64_t)splits * parts; }
  uint64_t sums_bytes(uint32_t N, uint32_t K) const { return pieces() > 1 ? (pieces() * N * K * 4 + 15) & ~15ull : 0; }
};

Plan plan_of(uint64_t T, uint32_t N, uint32_t K, int dy_dtype, bool aligned) {
  Plan p;
  p.parts = dy_dtype == IBP_BF16 ? 1 : dy_dtype == IBP_F16 ? 2 : 3;
  const uint64_t big = (((uint64_t)N + 255) / 256) * (((uint64_t)K + 255) / 256);
  // a short product costs less than the copy (11137 tokens of 3825: 200 inputs 60 us against
  // 75, 299 inputs 93 against 87, 2400 inputs 557 against 291)
  p.copied = p.parts > 1 || (N % 8 != 0 && K > 256);
  // BF16 rows of whole pieces that begin off 16 bytes take the small tile, through registers:
  // its ranges are as many or fewer, so the workspace is large enough for both.  Without tokens
  // there is nothing to lay out, and the small tile writes the zeros.
  p.big = T > 0 && (big > 128 || (T >= 3500 && big * T >= 140000)) && (p.copied || (aligned && N % 8 == 0));
  p.copied = p.copied && p.big;
  const uint32_t wide = p.big ? 256 : 128;
  p.tiles_o = (uint32_t)(((uint64_t)N + wide - 1) / wide);
  p.tiles_i = (uint32_t)(((uint64_t)K + wide - 1) / wide);
  const uint64_t tiles = (uint64_t)p.tiles_o * p.tiles_i, least = p.big ? 512 : 256;
  const uint64_t want = 256 / (tiles * p.parts), most = (T + least - 1) / least;
  uint64_t n = want < most ? want : most;
  n = n < 1 ? 1 : (n > 32 ? 32 : n);
  p.t_each = ((T + n - 1) / n + kT - 1) / kT * kT;
  if (p.t_each == 0) p.t_each = kT;
  p.splits = T ? (uint32_t)((T + p.t_each - 1) / p.t_each) : 1;
  return p;
}

uint32_t padded(uint32_t N) { return (N + 7) / 8 * 8; }

template <int DO> hipError_t go(const MxWgradArgs &a, const Plan &p, void *dst, hipStream_t s) {
  const dim3 grid(p.tiles_o * p.tiles_i, p.splits * p.parts);
  auto launch = [&](auto kernel, uint32_t threads) {
    kernel<<<grid, threads, 0, s>>>(a, dst, p.t_each, p.tiles_o, p.tiles_i, p.splits);
    return hipGetLastError();
  };
  if (p.big) return launch(wgrad_kernel<16, 2, 4, 8, 4, true, IBP_BF16, DO>, 512);
  if constexpr (DO == IBP_F32) {  // parts are always joined
    if (a.dy_dtype == IBP_F16) return launch(wgrad_kernel<32, 2, 2, 2, 2, false, IBP_F16, DO>, 256);
    if (a.dy_dtype == IBP_F32) return launch(wgrad_kernel<32, 2, 2, 2, 2, false, IBP_F32, DO>, 256);
  }
  return a.N % 8 == 0 && (uintptr_t)a.dy % 16 == 0 ? launch(wgrad_kernel<32, 2, 2, 2, 2, true, IBP_BF16, DO>, 256)
                                                   : launch(wgrad_kernel<32, 2, 2, 2, 2, false, IBP_BF16, DO>, 256);
}

}  // namespace

uint64_t mx_wgrad_workspace(uint64_t T, uint32_t N, uint32_t K, int dy_dtype) {
  const Plan p = plan_of(T, N, K, dy_dtype, true);
  return p.sums_bytes(N, K) + (p.copied ? p.parts * T * padded(N) * 2 : 0);
}

hipError_t launch_mx_wgrad(const MxWgradArgs &args, hipStream_t s) {
  MxWgradArgs a = args;
  const Plan p = plan_of(a.T, a.N, a.K, a.dy_dtype, (uintptr_t)a.dy % 16 == 0);
  if (p.t_each > 0x7FFFFFFFull) return hipErrorInvalidValue;
  a.dy_pitch = a.N;
  if (p.copied) {
    a.dy_pitch = padded(a.N);
    __bf16 *copy = reinterpret_cast<__bf16 *>(reinterpret_cast<uint8_t *>(a.ws) + p.sums_bytes(a.N, a.K));
    const uint64_t n = (a.T * (a.dy_pitch / 8) + kBlock - 1) / kBlock;
    const hipError_t e = with_dtype(a.dy_dtype, [&](auto d) {
      wgrad_parts_kernel<d.value><<<(uint32_t)(n < (1u << 20) ? n : (1u << 20)), kBlock, 0, s>>>(a, copy, p.parts);
      return hipGetLastError();
    });
    if (e != hipSuccess) return e;
    a.dy = copy;
  }
  if (p.pieces() > 1) {
    const hipError_t e = go<IBP_F32>(a, p, a.ws, s);
    if (e != hipSuccess) return e;
  }
  return with_dtype(a.dtype, [&](auto d) {
    if (p.pieces() == 1) return go<d.value>(a, p, a.dw, s);
    const uint64_t n = ((uint64_t)a.N * a.K + kBlock * 4 - 1) / (kBlock * 4);
    wgrad_join_kernel<d.value><<<(uint32_t)(n < 4096 ? n : 4096), kBlock, 0, s>>>(a, (uint32_t)p.pieces());
    return hipGetLastError();
  });
}

}  // namespace ibp
