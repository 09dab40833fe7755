// ibp_tile.h -- what the matrix products share: direct global-to-LDS loads, operand tiles
// of byte codes in LDS, the order in which output tiles are given to workgroups, and the
// search for the expert that a unit of grouped rows belongs to.
#pragma once

#include "ibp_device.h"
#include "ibp_num.h"

namespace ibp {
namespace dev {

// Source of the loads that stand for bytes past a row's or a matrix's end, as long as the
// longest of them (eight floats).
static __device__ __align__(32) const uint8_t kZeros[32] = {};

typedef __attribute__((address_space(3))) void lds_void;
typedef const __attribute__((address_space(1))) void global_void;

// Lane l's 16 bytes at `from` go to byte 16 l of the wavefront's `to`.
__device__ __forceinline__ void to_lds16(const uint8_t *from, uint8_t *to) {
  __builtin_amdgcn_global_load_lds((global_void *)from, (lds_void *)to, 16, 0, 0);
}

// A load that the compiler knows to be of global memory: from a pointer chosen between a
// matrix and kZeros it would make a flat load, which LDS waits count too.
template <typename T> __device__ __forceinline__ T from_global(const uint8_t *p) {
  return *reinterpret_cast<const __attribute__((address_space(1))) T *>((uintptr_t)p);
}

// Tile of a workgroup among rows x cols of them.  Workgroups go to the eight XCDs in
// turn; the tiles of one XCD lie together, in bands of kBand tile rows walked column by
// column, so its L2 keeps the band's rows.
struct TileId { uint32_t row, col; };
__device__ __forceinline__ TileId tile_of(uint32_t block, uint32_t rows, uint32_t cols) {
  constexpr uint32_t kXcds = 8, kBand = 8;
  const uint32_t total = rows * cols, per = total / kXcds, rest = total % kXcds;
  const uint32_t x = block % kXcds;
  const uint32_t id = x * per + (x < rest ? x : rest) + block / kXcds;
  const uint32_t band = id / (kBand * cols), in = id % (kBand * cols);
  const uint32_t high = rows - band * kBand < kBand ? rows - band * kBand : kBand;
  return TileId{band * kBand + in % high, in / high};
}

// A 16-byte piece of a row, zero from byte `pitch` on.
__device__ __forceinline__ uint4 piece(const uint8_t *row, uint32_t at, uint32_t pitch) {
  return at < pitch ? *reinterpret_cast<const uint4 *>(row + at) : make_uint4(0u, 0u, 0u, 0u);
}

// LDS rows of a stage are PITCH = 128 or 64 bytes.  The 16-byte pieces of a row are permuted by
// the row number, so that eight rows read at one piece lie in different banks: a read takes 4
// clocks then, 256 bytes a clock (measured; 8 with (row >> 2) & 3 for 64-byte rows, 8 and 16
// with none).  The loads write LDS in lane order, so the lanes' sources make the permutation.
template <uint32_t PITCH> __device__ __forceinline__ uint32_t swizzle(uint32_t row, uint32_t piece) {
  return piece ^ (PITCH == 128 ? row & 7 : (row >> 1) & 3);
}

// One operand's codes of a stage: ROWS rows of PITCH bytes, the loads shared by WAVES wavefronts.
template <uint32_t ROWS, uint32_t PITCH, uint32_t WAVES> struct Tile {
  static constexpr uint32_t kBytes = ROWS * PITCH, kLoads = kBytes / (1024 * WAVES);
  static_assert(WAVES * 1024 / PITCH % 8 == 0, "the permutation is the same for all of a lane's pieces");
  const uint8_t *code[kLoads];
  uint32_t at;

  __device__ __forceinline__ void init(const uint8_t *codes, uint64_t row0, uint64_t rows, uint32_t cp, uint32_t wave,
                                       uint32_t lane) {
    const uint32_t first = (wave * 64 + lane) / (PITCH / 16);
    at = swizzle<PITCH>(first, lane % (PITCH / 16)) * 16;
#pragma unroll
    for (uint32_t i = 0; i < kLoads; ++i) {
      const uint32_t row = i * (WAVES * 1024 / PITCH) + first;
      const uint64_t r = row0 + row < rows ? row0 + row : rows - 1;  // results of rows past the end are not stored
      code[i] = codes + r * cp + at;
    }
  }
  // The rows' bytes from k on, zeros past the rows' ends.
  __device__ __forceinline__ void load(uint8_t *lds, uint32_t k, uint32_t cp, uint32_t wave) {
#pragma unroll
    for (uint32_t i = 0; i < kLoads; ++i)
      to_lds16(k + at < cp ? code[i] + k : kZeros, lds + (i * WAVES + wave) * 1024);
  }
};

// A barrier that the compiler moves nothing across.
__device__ __forceinline__ void phase_barrier() {
  asm volatile("" ::: "memory");
  __builtin_amdgcn_sched_barrier(0);
  __builtin_amdgcn_s_barrier();
  __builtin_amdgcn_sched_barrier(0);
  asm volatile("" ::: "memory");
}

// A wavefront's FM x FN fragments, value(m, n) being four consecutive columns of a lane's row
// of fragment (m, n), into y from row0 and col0 on, rows and columns below their ends (at most
// 2^30).  They go through LDS (`out`, the wavefront's own), AT fragments' rows at a time, so that
// a store covers whole lines of y (from the fragments themselves a row gets 32 bytes at a time).
// STREAM: past the caches, which large results would empty of operands (the weight gradients of 32
// experts, 2048 x 4096, 537 MB: of 32768 tokens 563 us without, 533 with; of 8192 254 and 214;
// the product of 32768 rows, 134 MB, and the packing that reads it 430 and 422; that of 8-bit
// integers, 134 MB, 235 and 239).  Small results gain too, also where the next operator reads them
// at once (product and packing of 4096 rows of 8 experts, 1024 x 1024, 8 MB: e4m3 24.4 and 22.7,
// e2m1 17.0 and 15.5), but not the gradients of few tokens (2500 of 45 experts, 500 x 600, 27 MB:
// 24.4 and 25.2; 54 MB: 27.4 and 30.7).
template <typename TO, int FN, int AT = 2> constexpr uint32_t out_bytes() { return AT * 16 * (16 * FN * sizeof(TO) + 16); }
template <typename TO, int FM, int FN, int AT = 2, bool STREAM = false, typename F>
__device__ __forceinline__ void store_fragments(TO *out, TO *y, uint32_t row0, uint32_t rows, uint32_t col0,
                                                uint32_t cols, uint32_t lane, F &&value) {
  constexpr uint32_t kCols = 16 * FN, kPad = 16 / sizeof(TO), kEach = 16 / sizeof(TO), kPieces = AT * 16 * kCols / kEach / 64;
  typedef TO Aligned __attribute__((ext_vector_type(kEach)));
  typedef TO Loose __attribute__((ext_vector_type(kEach), aligned(sizeof(TO))));
  typedef TO Four __attribute__((ext_vector_type(4)));
  const uint32_t r = lane & 15, g = lane >> 4;
#pragma unroll
  for (int m = 0; m < FM; m += AT) {
    wave_lds_sync();
#pragma unroll
    for (int h = 0; h < AT; ++h)
#pragma unroll
      for (int n = 0; n < FN; ++n) {
        const v4f x = value(m + h, n);
        *reinterpret_cast<Four *>(out + (16 * h + r) * (kCols + kPad) + 16 * n + 4 * g) = Four{(TO)x[0], (TO)x[1], (TO)x[2], (TO)x[3]};
      }
    wave_lds_sync();
#pragma unroll
    for (uint32_t p = 0; p < kPieces; ++p) {
      const uint32_t slot = p * 64 + lane, row = slot / (kCols / kEach), c = slot % (kCols / kEach) * kEach;
      const uint32_t gm = row0 + 16 * m + row, gn = col0 + c;
      if (gm >= rows || gn >= cols) continue;
      const Aligned x = *reinterpret_cast<const Aligned *>(out + row * (kCols + kPad) + c);
      if (gn + kEach <= cols) {
        if constexpr (STREAM) __builtin_nontemporal_store((Loose)x, reinterpret_cast<Loose *>(y + (uint64_t)gm * cols + gn));
        else *reinterpret_cast<Loose *>(y + (uint64_t)gm * cols + gn) = x;
      } else {
#pragma unroll
        for (uint32_t e = 0; e < kEach; ++e)
          if (gn + e < cols) y[(uint64_t)gm * cols + gn + e] = x[e];
      }
    }
  }
}

// Rows sorted by expert: rows [offsets[e], offsets[e + 1]) are expert e's, cut into units of
// `1 << shift` rows, experts in order.  What the offsets say is held within the rows that
// there are, so bad ones lead nowhere outside.  Each wavefront searches by itself, a lane for
// every 64th part of the experts: offsets are on the device, and a list made by a launch of
// its own would cost more than the search.
struct Experts {
  const int64_t *offsets;
  uint32_t n;       // experts
  uint32_t shift;   // log2 of the rows of a unit
  uint64_t rows;    // of all experts

  __device__ __forceinline__ uint64_t start(uint32_t e) const {
    const int64_t o = offsets[e];
    return o < 0 ? 0 : ((uint64_t)o < rows ? (uint64_t)o : rows);
  }
};

struct Unit {
  uint32_t expert;
  uint64_t row0, begin, end;  // the unit's first row; its expert's rows
};

// EMPTY: an expert without rows has one unit all the same.
template <bool EMPTY> struct UnitSearch {
  Experts x;
  uint32_t per, before, mine, total;  // experts a lane; units of lanes before, of this one, of all

  __device__ __forceinline__ uint32_t units(uint64_t b, uint64_t e) const {
    const uint32_t u = e > b ? (uint32_t)((e - b + (1ull << x.shift) - 1) >> x.shift) : 0u;
    return EMPTY && u == 0 ? 1u : u;
  }
  __device__ __forceinline__ UnitSearch(const Experts &experts) : x(experts) {
    per = (x.n + kWave - 1) / kWave;
    const uint32_t e0 = lane_id() * per;
    mine = 0;
    for (uint32_t e = e0; e < e0 + per && e < x.n; ++e) mine += units(x.start(e), x.start(e + 1));
    const uint32_t incl = wave_incl_scan(mine);
    before = incl - mine;
    total = (uint32_t)__builtin_amdgcn_readlane((int)incl, kWave - 1);
  }
  // An expert's first unit and how many it has.
  __device__ __forceinline__ uint2 units_of(uint32_t expert) const {
    const uint32_t e0 = lane_id() * per;
    uint32_t first = before;
    for (uint32_t e = e0; e < e0 + per && e < expert; ++e) first += units(x.start(e), x.start(e + 1));
    first = (uint32_t)__builtin_amdgcn_readlane((int)first, (int)(expert / per));
    return make_uint2(first, units(x.start(expert), x.start(expert + 1)));
  }
  // Unit u < total.
  __device__ __forceinline__ Unit find(uint32_t u) const {
    uint32_t left = u - before, e = lane_id() * per;
    uint64_t b = 0, end = 0;
    const bool own = u >= before && left < mine;
    if (own) {
      const uint32_t last = (e + per < x.n ? e + per : x.n) - 1;
      for (;; ++e) {
        b = x.start(e);
        end = x.start(e + 1);
        const uint32_t k = units(b, end);
        if (left < k || e == last) break;
        left -= k;
      }
      if (end < b) end = b;
    }
    const int lane = __builtin_ctzll(ballot(own) | 1ull << 63);
    auto get = [&](uint32_t v) { return (uint32_t)__builtin_amdgcn_readlane((int)v, lane); };
    auto get64 = [&](uint64_t v) { return (uint64_t)get((uint32_t)(v >> 32)) << 32 | get((uint32_t)v); };
    Unit r;
    r.expert = get(e);
    r.begin = get64(b);
    r.end = get64(end);
    r.row0 = r.begin + ((uint64_t)get(left) << x.shift);
    return r;
  }
};

// The expert that comes `place`th by its rows, the most first, of up to a wavefront's lanes of
// experts with less than 2^32 rows: of the sizes' bits from the highest on, those with the bit
// come before those without.
__device__ __forceinline__ uint32_t by_size(const Experts &x, uint32_t place) {
  const uint32_t e = lane_id();
  uint32_t size = 0;
  if (e < x.n) {
    const uint64_t b = x.start(e), end = x.start(e + 1);
    size = end > b ? (uint32_t)(end - b) : 0u;
  }
  uint64_t left = ~0ull >> (kWave - x.n);
  for (uint32_t bits = 64 - (uint32_t)__builtin_clzll(x.rows | 1); bits > 0; --bits) {
    const uint64_t more = ballot(size >> (bits - 1) & 1) & left;
    const uint32_t n = popc(more);
    const bool among = place < n;
    left = among ? more : left & ~more;
    place -= among ? 0u : n;
  }
  return (uint32_t)__builtin_ctzll(ballot((left >> e & 1) && count_below(left) == place));
}

// Offsets that fall or leave the rows, seen by the calling wavefront's lanes together.
__device__ __forceinline__ void check_offsets(const Experts &x, uint32_t *err) {
  bool bad = false;
  for (uint32_t e = lane_id(); e < x.n; e += kWave) {
    const int64_t b = x.offsets[e], n = x.offsets[e + 1];
    bad = bad || b < 0 || n < b || (uint64_t)n > x.rows;
  }
  if (ballot(bad) && lane_id() == 0) atomicOr(err, (uint32_t)IBP_DEVERR_CORRUPT);
}

}  // namespace dev

// Most units of `1 << shift` of `rows` rows that experts can have: each expert with rows one
// that its last row ends, and what is left in whole ones; with `empty` each of the others too.
inline uint64_t most_units(uint64_t rows, uint64_t experts, uint32_t shift, bool empty) {
  const uint64_t used = rows < experts ? rows : experts;
  return empty ? (rows >> shift) + experts : ((rows - used) >> shift) + used;
}

}  // namespace ibp
