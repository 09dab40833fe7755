// ibp_tile.h -- what the matrix products share: direct global-to-LDS loads and the order
// in which output tiles are given to workgroups.
#pragma once

#include "ibp_device.h"

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

}  // namespace dev
}  // namespace ibp
