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
// where the result is not.  Each step is rounded to 32 bits, and then the result to y's type, in
// every kernel here alike.
__device__ __forceinline__ float scaled(int sum, float sa, float sb) {
  const bool a_less = fabsf(sa) < fabsf(sb);
  return (float)sum * (a_less ? sa : sb) * (a_less ? sb : sa);
}

__device__ __forceinline__ v4f scaled4(v4i sum, float sa, v4f sb) {
  return as_floats(v4f{scaled(sum[0], sa, sb[0]), scaled(sum[1], sa, sb[1]), scaled(sum[2], sa, sb[2]), scaled(sum[3], sa, sb[3])});
}

// Few rows of A.  A workgroup computes 16 x 16 outputs, its wavefronts take steps of 256 codes
// in turn and their sums are added through LDS.  Bound by reading the weights: one row by
// 8192 outputs, 8192 deep takes 13.6 us, 4.9 TB/s.  (With the next step's loads in flight it
// takes 14.3, and 4096 x 4096 7.1 instead of 5.5: twice the registers, half the wavefronts.)
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
               scaled4(acc, a.a_scales[m0 + r], load4(a.b_scales, n0 + 4 * g, a.N)));
}

hipError_t go_direct(const I8MatmulArgs &a, hipStream_t s) {
  const uint64_t gx = (a.N + 15) / 16, gy = (a.M + 15) / 16;
  const uint32_t steps = (a.K + kStep - 1) / kStep;
  // Up to one workgroup a CU eight wavefronts, which share a long k (one row by 4096 outputs,
  // 14336 deep: 11.6 us, four 15.9, sixteen 12.6); beyond, four (8192 x 8192: 13.8, eight 14.7).
  uint32_t waves = gx * gy <= 256 ? 8 : 4;
  while (waves > 1 && waves > steps) waves /= 2;
  return with_dtype(a.dtype, [&](auto d) {
    i8_direct_kernel<d.value><<<dim3((uint32_t)gx, (uint32_t)gy), waves * kWave, (waves - 1) * 1024, s>>>(a);
    return hipGetLastError();
  });
}

// ------------------------------------------------------------------ many rows

// A workgroup of WM x WN wavefronts computes 16 FM WM rows of A by 16 FN WN rows of B over
// stages_each stages of k, from blockIdx.y * stages_each on: outputs, or with SUMS the sums
// into a.ws + blockIdx.y * M * N.
//
// Operands go through LDS by the direct global-to-LDS loads, in stages of 128 codes of every
// row; a stage is two units, A's rows and B's, in a ring of UNITS units, and two matrix
// instructions deep.  128 bytes of a row are a whole line of memory: loads of 64 fill LDS at 14
// TB/s, of 128 at 22 (measured without the rest).
//
// Four wavefronts have one barrier a stage.  Eight, two a SIMD, take each half of a stage in a
// reading phase and a multiplying phase with a barrier after each; the second half of the
// wavefronts runs one phase behind the first, so LDS serves one half while the other
// multiplies.  They go on from tile to tile, and a tile's results leave while the next one's
// first stages arrive (8192 x 8192 outputs, 512 deep: 55.5 us, 59.0 without; 4096 deep 232 and
// 235).  8192 x 8192 x 4096 takes 232 us, 2.4 POP/s, 8192 deep 429, 2.6 (registers alone reach
// 3.5 with such operands, 4.5 with zeros): bound by power (194 us with zeros) and by the phases,
// matrix units busy 54% of the time.  In turn with the library's product of 8-bit integers to
// 32-bit sums: 230 us against 241, 4096 x 4096 x 4096 60 against 64, 1024 x 4096 x 4096 28 against 25.
template <int WM, int WN, int FM, int FN, uint32_t UNITS, bool SUMS, int DO>
__global__ __launch_bounds__(WM *WN *64, 2) void i8_tile_kernel(I8MatmulArgs a, uint32_t tiles_m, uint32_t tiles_n,
                                                             uint32_t stages_each) {
  using TO = typename Num<DO>::T;
  constexpr uint32_t kWaves = WM * WN, kRowsA = 16 * FM * WM, kRowsB = 16 * FN * WN, kPitch = 128;
  using TileA = Tile<kRowsA, kPitch, kWaves>;
  using TileB = Tile<kRowsB, kPitch, kWaves>;
  static_assert(kRowsA == kRowsB, "units have one size");
  constexpr uint32_t kUnit = TileA::kBytes, kLoads = TileA::kLoads;  // a wavefront's loads per unit
  static_assert(UNITS >= 5 && UNITS * kUnit <= 160 * 1024 && (UNITS - 2) * kLoads < 64, "");
  __shared__ __align__(1024) uint8_t ring[UNITS * kUnit];
  const uint32_t lane = lane_id(), wave = uniform(threadIdx.x / kWave), r = lane & 15, g = lane >> 4;
  const uint32_t cp = (uint32_t)i8_pitch(a.K);
  uint32_t m0, n0;  // rows are at most 2^30
  TileA ta;
  TileB tb;
  auto aim = [&](uint32_t tile) {
    const TileId t = tile_of(tile, tiles_m, tiles_n);
    m0 = t.row * kRowsA;
    n0 = t.col * kRowsB;
    ta.init(a.a_codes, m0, a.M, cp, wave, lane);
    tb.init(a.b_codes, n0, a.N, cp, wave, lane);
  };
  aim(blockIdx.x);
  const uint32_t wm = (wave % WM) * 16 * FM, wn = (wave / WM) * 16 * FN;
  v4i acc[FN][FM];
  auto clear = [&] {
#pragma unroll
    for (int n = 0; n < FN; ++n)
#pragma unroll
      for (int m = 0; m < FM; ++m) acc[n][m] = v4i{0, 0, 0, 0};
  };

  const uint32_t all = (cp + kPitch - 1) / kPitch, begin = blockIdx.y * stages_each;
  const uint32_t steps = all - begin < stages_each ? all - begin : stages_each;
  // Units are loaded in order, A's rows of a stage and B's, into one place of the ring after
  // another.  Always kLoads loads, of zeros past the rows' end: the waits below count on it.
  uint32_t fill_at = 0;
  auto place_after = [](uint32_t at, uint32_t units) { return at + units * kUnit >= UNITS * kUnit ? at + units * kUnit - UNITS * kUnit : at + units * kUnit; };
  auto fill = [&](bool of_b, uint32_t stage) {
    const uint32_t k = (begin + stage) * kPitch;
    if (of_b) tb.load(ring + fill_at, k, cp, wave);
    else ta.load(ring + fill_at, k, cp, wave);
    fill_at = place_after(fill_at, 1);
  };
  // The two units that take the places of stage s: B's of one stage, A's of the next, or both of one.
  auto refill = [&](uint32_t s) {
    fill(UNITS % 2, s + UNITS / 2);
    fill(!(UNITS % 2), s + (UNITS + 1) / 2);
  };
  // a fragment's rows are 16 apart and its permutation goes by r alone: one address, then offsets
  uint32_t at_a[2], at_b[2];
#pragma unroll
  for (uint32_t h = 0; h < 2; ++h) {
    at_a[h] = (wm + r) * kPitch + swizzle<kPitch>(r, 4 * h + g) * 16;
    at_b[h] = (wn + r) * kPitch + swizzle<kPitch>(r, 4 * h + g) * 16;
  }
  struct Half {  // fragments of one half of a stage
    v4i w[FN], v[FM];
  };
  // What is filled is not what is read; __restrict__ says so to the compiler, which
  // otherwise would wait for all loads in flight before an LDS read.
  auto read = [&](Half &f, uint8_t *__restrict__ filled, const uint8_t *__restrict__ ua, const uint8_t *__restrict__ ub, uint32_t h) {
    (void)filled;
#pragma unroll
    for (int n = 0; n < FN; ++n) f.w[n] = *reinterpret_cast<const v4i *>(ub + at_b[h] + n * 16 * kPitch);
#pragma unroll
    for (int m = 0; m < FM; ++m) f.v[m] = *reinterpret_cast<const v4i *>(ua + at_a[h] + m * 16 * kPitch);
  };
  constexpr bool kPingPong = kWaves == 8;
#pragma unroll
  for (uint32_t u = 0; u < UNITS - (kPingPong ? 0 : 2); ++u) fill(u % 2, u / 2);
  // All loads but those of the units behind the next stage.
  constexpr int kNext = wait_loads_and_lds((UNITS - 4) * kLoads);
  uint32_t now = 0;  // place of stage s's first unit
  if constexpr (kPingPong) {
    static_assert(!SUMS && UNITS == 5, "");
    const bool behind = wave >= kWaves / 2;
    // Results go through the last two places of the ring while the next tile's first three
    // units are on their way into the others.
    constexpr int kAt = sizeof(TO) == 2 ? 2 : 1;
    static_assert(kWaves * out_bytes<TO, FN, kAt>() <= 2 * kUnit, "");
    constexpr uint32_t kStores = FM * 16 * 16 * FN * sizeof(TO) / 1024;  // of a wavefront, of a whole tile
    static_assert(3 * kLoads + kStores < 64, "");
    __builtin_amdgcn_s_waitcnt(wait_loads_and_lds((UNITS - 2) * kLoads));
    for (uint32_t tile = blockIdx.x;;) {
      clear();
      phase_barrier();
      if (behind) phase_barrier();
#pragma unroll 1
      for (uint32_t s = 0; s < steps; ++s) {
        const uint32_t now_b = place_after(now, 1);
#pragma unroll
        for (uint32_t h = 0; h < 2; ++h) {
          Half f;
          read(f, ring + fill_at, ring + now, ring + now_b, h);
          // These reads are done; in the last phase before the first half reads stage s + 1, so
          // are every wavefront's loads of it, but not those of the units after it.
          __builtin_amdgcn_s_waitcnt(0xC07F);
          if (h == 1 && behind) __builtin_amdgcn_s_waitcnt(kNext);
          phase_barrier();
          __builtin_amdgcn_s_setprio(1);
#pragma unroll
          for (int m = 0; m < FM; ++m) {
#pragma unroll
            for (int n = 0; n < FN; ++n) acc[n][m] = mfma(f.w[n], f.v[m], acc[n][m]);
            if (m == 0) {
              // The places of a stage that all have read: the half behind has when it multiplies the
              // second half of it, the other when it multiplies the first of the next.
              __builtin_amdgcn_sched_barrier(0);  // the compiler would issue the loads first
              if (behind ? h == 1 : h == 0 && s > 0) refill(behind ? s : s - 1);
            }
          }
          __builtin_amdgcn_sched_barrier(0);
          __builtin_amdgcn_s_setprio(0);
          if (h == 1 && !behind) __builtin_amdgcn_s_waitcnt(kNext);
          phase_barrier();
        }
        now = place_after(now, 2);
      }
      if (!behind) phase_barrier();
      const uint32_t row0 = m0 + wm, col0 = n0 + wn;
      const bool whole = m0 + kRowsA <= a.M && n0 + kRowsB <= a.N;
      v4f sb[FN];
      float sa[FM];
#pragma unroll
      for (int n = 0; n < FN; ++n) sb[n] = load4(a.b_scales, col0 + 16 * n + 4 * g, a.N);
#pragma unroll
      for (int m = 0; m < FM; ++m) sa[m] = row0 + 16 * m + r < a.M ? a.a_scales[row0 + 16 * m + r] : 0.0f;
      __builtin_amdgcn_s_waitcnt(kWaitVmcnt0);  // these, and the loads into LDS past the last stage
      phase_barrier();
      tile += gridDim.x;
      const bool more = tile < tiles_m * tiles_n;
      now = fill_at = 0;
      if (more) {
        aim(tile);
#pragma unroll
        for (uint32_t u = 0; u < 3; ++u) fill(u % 2, u / 2);
      }
      store_fragments<TO, FM, FN, kAt>(reinterpret_cast<TO *>(ring + 3 * kUnit + wave * out_bytes<TO, FN, kAt>()),
                                       static_cast<TO *>(a.y), row0, (uint32_t)a.M, col0, (uint32_t)a.N, lane,
                                       [&](int m, int n) { return scaled4(acc[n][m], sa[m], sb[n]); });
      if (!more) return;
      phase_barrier();  // all have stored
#pragma unroll
      for (uint32_t u = 3; u < UNITS; ++u) fill(u % 2, u / 2);
      // Stage 0 is there; what was asked for later is one unit, the stores and two units.
      if (whole) __builtin_amdgcn_s_waitcnt(wait_loads_and_lds(3 * kLoads + kStores));
      else __builtin_amdgcn_s_waitcnt(wait_loads_and_lds(3 * kLoads));
    }
  } else {
    clear();
    // One barrier a stage: every wavefront's loads of it are done, and all have read the stage
    // before, whose places are filled anew.
#pragma unroll 1
    for (uint32_t s = 0; s < steps; ++s) {
      __builtin_amdgcn_s_waitcnt(kNext);
      phase_barrier();
      Half f[2];
      uint8_t *const filled = ring + fill_at;
#pragma unroll
      for (uint32_t h = 0; h < 2; ++h) read(f[h], filled, ring + now, ring + place_after(now, 1), h);
      __builtin_amdgcn_sched_barrier(0);
      refill(s - 1);
#pragma unroll
      for (uint32_t h = 0; h < 2; ++h) {
        __builtin_amdgcn_sched_barrier(0);
#pragma unroll
        for (int m = 0; m < FM; ++m)
#pragma unroll
          for (int n = 0; n < FN; ++n) acc[n][m] = mfma(f[h].w[n], f[h].v[m], acc[n][m]);
      }
      __builtin_amdgcn_sched_barrier(0);
      now = place_after(now, 2);
    }
  }
  __builtin_amdgcn_s_waitcnt(kWaitVmcnt0);  // no load into LDS outlives the workgroup
  __syncthreads();
  if constexpr (SUMS) {
    int32_t *ws = a.ws + (uint64_t)blockIdx.y * a.M * a.N;
#pragma unroll
    for (int m = 0; m < FM; ++m) {
      const uint64_t gm = m0 + wm + 16 * m + r;
      if (gm >= a.M) continue;
#pragma unroll
      for (int n = 0; n < FN; ++n) {
        const uint64_t gn = n0 + wn + 16 * n + 4 * g;
        typedef int V __attribute__((ext_vector_type(4), aligned(4)));
        if (gn + 4 <= a.N) {
          *reinterpret_cast<V *>(ws + gm * a.N + gn) = acc[n][m];
        } else {
#pragma unroll
          for (int i = 0; i < 4; ++i)
            if (gn + i < a.N) ws[gm * a.N + gn + i] = acc[n][m][i];
        }
      }
    }
  } else {
    static_assert(kWaves * out_bytes<TO, FN>() <= sizeof(ring), "");
    v4f sb[FN];
    float sa[FM];
#pragma unroll
    for (int n = 0; n < FN; ++n) sb[n] = load4(a.b_scales, n0 + wn + 16 * n + 4 * g, a.N);
#pragma unroll
    for (int m = 0; m < FM; ++m) sa[m] = m0 + wm + 16 * m + r < a.M ? a.a_scales[m0 + wm + 16 * m + r] : 0.0f;
    store_fragments<TO, FM, FN>(reinterpret_cast<TO *>(ring + wave * out_bytes<TO, FN>()), static_cast<TO *>(a.y), m0 + wm,
                                (uint32_t)a.M, n0 + wn, (uint32_t)a.N, lane, [&](int m, int n) { return scaled4(acc[n][m], sa[m], sb[n]); });
  }
}

// Adds the ranges' sums, and scales them.
template <int DO> __global__ __launch_bounds__(kBlock) void i8_join_kernel(I8MatmulArgs a, uint32_t splits) {
  using TO = typename Num<DO>::T;
  const uint64_t m = blockIdx.y, n = a.M * a.N;
  for (uint64_t c = ((uint64_t)blockIdx.x * kBlock + threadIdx.x) * 4; c < a.N; c += (uint64_t)gridDim.x * kBlock * 4) {
    v4i s{0, 0, 0, 0};
    typedef int V __attribute__((ext_vector_type(4), aligned(4)));
    for (uint32_t k = 0; k < splits; ++k) {
      const int32_t *from = a.ws + k * n + m * a.N + c;
      if (c + 4 <= a.N) {
        s += (v4i)*reinterpret_cast<const V *>(from);
      } else {
        for (int i = 0; i < 4; ++i)
          if (c + i < a.N) s[i] += from[i];
      }
    }
    store4<TO>(static_cast<TO *>(a.y) + m * a.N, c, a.N, scaled4(s, a.a_scales[m], load4(a.b_scales, c, a.N)));
  }
}

// Which kernel, and how often k is cut.
struct Plan {
  enum Kind { kDirect, kSmall, kMiddle, kBig } kind;
  uint32_t tiles_m, tiles_n, splits, stages_each;
};

Plan plan_of(uint64_t M, uint64_t N, uint32_t K) {
  Plan p{Plan::kDirect, 0, 0, 1, 1};
  // A few rows, which have only the weights to read (8192 x 8192 weights: 8 rows 15.0 us, small
  // tiles 14.9; 16 rows 17.6, 14.9), or so little work that a workgroup has a few steps (64 x
  // 2048 outputs, 2048 deep 6.2 us against 6.8; 32 x 4096, 4096 deep 9.9 against 9.4; 1000 x
  // 1000, 64 deep 4.3 against 3.8).
  const uint64_t blocks = ((M + 15) / 16) * ((N + 15) / 16);
  if ((M <= 8 && blocks <= 1u << 22) || (blocks <= 1024 && blocks * K <= 1u << 20)) return p;
  auto tiles = [&](uint64_t wide) { return ((M + wide - 1) / wide) * ((N + wide - 1) / wide); };
  const uint64_t least = M < N ? M : N;
  // Larger tiles read each operand less often, smaller ones are more and finish a stage
  // sooner.  64 x 64: 1024 x 2048 outputs (128 tiles of 128), 4096 deep 15.4 us against 24.9 with
  // 128 x 128; 1500 x 2000 (192), 1000 deep 10.2 and 10.7; 1024 x 4096 (256), 4096 deep 28.9 and
  // 27.1; 64 x 65536 46.6 and 46.5, 100 x 65536 67.1 and 48.9.  256 x 256: 2048 x 4096 outputs
  // (128 tiles of 256), 2048 deep 33.0 against 28.7 with 128 x 128; 1536 x 8192 (192), 4096 deep
  // 56.6 and 63.8; 4096 x 4096 (256), 1024 deep 23.5 and 28.6; 256 x 32768 53.2 and 42.4.  A
  // launch holds less than 2^24 small tiles, each a workgroup; the others go on from tile to tile.
  p.kind = tiles(128) <= 192 || (least <= 64 && tiles(64) < 1u << 24) ? Plan::kSmall : (tiles(256) < 192 || least <= 256 ? Plan::kMiddle : Plan::kBig);
  const uint32_t wide = p.kind == Plan::kSmall ? 64 : (p.kind == Plan::kMiddle ? 128 : 256);
  p.tiles_m = (uint32_t)((M + wide - 1) / wide);
  p.tiles_n = (uint32_t)((N + wide - 1) / wide);
  // Where small tiles leave CUs empty, k is cut into ranges of at least 16 stages of 128 codes,
  // whose sums another launch adds (64 x 8192 outputs, 8192 deep: one range 20.3 us, two 16.0,
  // four 17.8; 333 x 1000, 2001 deep: 7.1, two ranges of 8 stages 8.5).
  const uint32_t stages = (uint32_t)((i8_pitch(K) + 127) / 128);
  const uint64_t want = p.kind == Plan::kSmall ? 256 / tiles(64) : 1, most = stages / 16;
  uint32_t n = (uint32_t)(want < most ? want : most);
  n = n < 1 ? 1 : (n > 8 ? 8 : n);
  p.stages_each = (stages + n - 1) / n;
  if (p.stages_each == 0) p.stages_each = 1;
  p.splits = stages ? (stages + p.stages_each - 1) / p.stages_each : 1;
  return p;
}

template <bool SUMS, int DO> hipError_t go_tile(const I8MatmulArgs &a, const Plan &p, hipStream_t s) {
  auto launch = [&](auto kernel, uint32_t threads, uint32_t most) {
    const uint32_t tiles = p.tiles_m * p.tiles_n;
    kernel<<<dim3(tiles < most ? tiles : most, p.splits), threads, 0, s>>>(a, p.tiles_m, p.tiles_n, p.stages_each);
  };
  // small tiles alone are cut; three workgroups of them, and two of the middle ones, fit a CU
  if (SUMS || p.kind == Plan::kSmall) launch(i8_tile_kernel<2, 2, 2, 2, 6, SUMS, DO>, 256, ~0u);
  else if constexpr (!SUMS) {
    if (p.kind == Plan::kMiddle) launch(i8_tile_kernel<2, 4, 4, 2, 5, false, DO>, 512, 512);
    else launch(i8_tile_kernel<2, 4, 8, 4, 5, false, DO>, 512, 256);
  }
  return hipGetLastError();
}

}  // namespace

uint64_t i8_matmul_workspace(uint64_t M, uint64_t N, uint32_t K) {
  const Plan p = plan_of(M, N, K);
  return p.splits > 1 ? p.splits * M * N * 4 : 0;
}

hipError_t launch_i8_matmul(const I8MatmulArgs &a, hipStream_t s) {
  const Plan p = plan_of(a.M, a.N, a.K);
  if (p.kind == Plan::kDirect) return go_direct(a, s);
  if (p.splits > 1) {
    const hipError_t e = go_tile<true, IBP_F32>(a, p, s);
    if (e != hipSuccess) return e;
  }
  return with_dtype(a.dtype, [&](auto d) {
    if (p.splits == 1) return go_tile<false, d.value>(a, p, s);
    const uint64_t n = (a.N + kBlock * 4 - 1) / (kBlock * 4);
    i8_join_kernel<d.value><<<dim3((uint32_t)(n < 64 ? n : 64), (uint32_t)a.M), kBlock, 0, s>>>(a, p.splits);
    return hipGetLastError();
  });
}

}  // namespace ibp
