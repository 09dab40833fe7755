// ibp_embed.hip -- embedding lookup with scaling, and its gradient by sorted tokens.
//
// Lookup: out[j] = scale * table[ids[j]], one read of each token's row and one write.
// Bound by HBM (65536 of 131072 rows of 4096 in bf16, frequent ids: 152 us, 7.1 TB/s of
// row reads and writes, rows that come again from cache); a lane moves eight elements,
// of four rows where there are enough.
//
// Gradient: grad[v] = scale * sum of dout[j] over the tokens j with ids[j] == v, in
// 32 bits, rows without tokens 0.  Tokens are sorted by id (stable, so a row's tokens
// keep their order and the sums do not depend on timing), the sorted list is cut into
// chunks of equal length, and each chunk's runs of equal ids are summed by one group of
// lanes: the work is even however unevenly the tokens fall on the rows.  A run that
// fills a chunk is cut at the chunks' borders; each piece leaves a 32-bit partial row,
// and a second kernel adds those.  dout is read once and grad written once; the sort
// moves 8 bytes a token a pass.  65536 tokens of 4096 in bf16, 131072 rows: 367 us, of
// which the sums and the rows without tokens take 332 (1.61 GB, 4.9 TB/s), the sort's
// four kernels 22, the cut runs 13.
#include "ibp_device.h"
#include "ibp_num.h"

namespace ibp {
namespace {

using namespace dev;

// ------------------------------------------------------------------ lookup

// Lanes that take a row: the smallest power of two that covers it, up to the workgroup.
uint32_t pow2_lanes(uint32_t dim) {
  uint32_t l = 1;
  while (l < (dim + 7) / 8 && l < kBlock) l *= 2;
  return l;
}

struct RowWalk {
  uint32_t lanes;   // lanes a row, a power of two up to kBlock
  uint32_t strips;  // workgroups that share a row's columns
  uint64_t units;   // strips of all groups of R * kBlock / lanes rows
};

template <int DI, int DO, uint32_t R> __global__ __launch_bounds__(kBlock) void lookup_kernel(LookupArgs a, RowWalk w) {
  using TI = typename Num<DI>::T;
  using TO = typename Num<DO>::T;
  const uint32_t tx = threadIdx.x & (w.lanes - 1), ty = threadIdx.x / w.lanes, rows_blk = kBlock / w.lanes;
  const TI *table = static_cast<const TI *>(a.table);
  TO *out = static_cast<TO *>(a.out);
  by_width(a.dim, [&](auto wide) {
    for (uint64_t unit = blockIdx.x; unit < w.units; unit += gridDim.x) {
      const uint64_t group = w.strips == 1 ? unit : unit / w.strips;
      const uint32_t c0 = ((uint32_t)(unit - group * w.strips) * w.lanes + tx) * 8;
      uint64_t row[R], id[R];
      int64_t v[R];
      bool ok[R];
#pragma unroll
      for (uint32_t k = 0; k < R; ++k) {
        row[k] = (group * R + k) * rows_blk + ty;
        v[k] = a.ids[row[k] < a.n_ids ? row[k] : a.n_ids - 1];
      }
#pragma unroll
      for (uint32_t k = 0; k < R; ++k) {
        ok[k] = v[k] >= 0 && (uint64_t)v[k] < a.n_rows;
        id[k] = ok[k] ? (uint64_t)v[k] : 0;
      }
      for (uint32_t c = c0; c < a.dim; c += w.strips * w.lanes * 8) {
        Vec8<TI> x[R];
#pragma unroll
        for (uint32_t k = 0; k < R; ++k) x[k] = load8<wide.value, TI>(table + id[k] * a.dim, c, a.dim);
#pragma unroll
        for (uint32_t k = 0; k < R; ++k) {
          if (row[k] >= a.n_ids) continue;
          F8 y = widen<wide.value, TI>(x[k], c, a.dim);
#pragma unroll
          for (int i = 0; i < 8; ++i) y.v[i] = ok[k] ? y.v[i] * a.scale : 0.0f;
          store8<TO>(out + row[k] * a.dim, c, a.dim, y);
        }
      }
      if (c0 == 0 && a.err) {
        bool bad = false;
#pragma unroll
        for (uint32_t k = 0; k < R; ++k) bad = bad || !ok[k];
        if (bad) atomicOr(a.err, IBP_DEVERR_BAD_ID);
      }
    }
  });
}

// ------------------------------------------------------------------ sort by id

// Radix sort of (key, position) pairs, keys 0..n_rows; key n_rows stands for tokens
// that take no part (the padding id, ids out of range) and sorts to the end.  Digits
// of up to nine bits: two passes cover 2^18 rows.
constexpr uint32_t kDigitBits = 9, kBins = 1u << kDigitBits;
constexpr uint32_t kSortBlocks = 256;     // at most this many workgroups a pass
constexpr uint32_t kSortMin = 1024;       // tokens per workgroup at least
constexpr uint32_t kSmallTokens = 8192;   // sorted by one workgroup in LDS
constexpr uint32_t kSortThreads = 1024, kSortWaves = kSortThreads / kWave;

struct Pair { uint32_t key, pos; };

struct SortArgs {
  const int64_t *ids;
  uint32_t *err;
  Pair *from, *to;      // from: unused by the first pass
  uint32_t *counts;     // [workgroup][kBins]
  uint32_t *crossing;   // [0] cleared for the sums: chunks listed
  uint64_t n_rows;
  int64_t padding_id;
  uint32_t n;
  uint32_t per_wave;    // tokens per wavefront, a multiple of kWave
  uint32_t shift, bits; // this pass's digit
};

__device__ __forceinline__ uint32_t key_of(const SortArgs &a, uint32_t j) {
  const int64_t v = a.ids[j];
  if (v == a.padding_id && v >= 0) return (uint32_t)a.n_rows;
  if (v < 0 || (uint64_t)v >= a.n_rows) {
    if (a.err) atomicOr(a.err, IBP_DEVERR_BAD_ID);
    return (uint32_t)a.n_rows;
  }
  return (uint32_t)v;
}

// Lanes of the wavefront whose digit equals this lane's, among the lanes of `live`.
__device__ __forceinline__ uint64_t same_digit(uint32_t d, uint32_t bits, uint64_t live) {
  uint64_t m = live;
  for (uint32_t b = 0; b < bits; ++b) {
    const uint64_t v = ballot((d >> b) & 1u);
    m &= (d >> b) & 1u ? v : ~v;
  }
  return m;
}

// Per workgroup, how many of its tokens have each digit.
template <bool FIRST> __global__ __launch_bounds__(kSortThreads) void sort_count_kernel(SortArgs a) {
  __shared__ uint32_t hist[kBins];
  if (threadIdx.x < kBins) hist[threadIdx.x] = 0;
  if constexpr (FIRST) {
    if (blockIdx.x == 0 && threadIdx.x == 0) a.crossing[0] = 0;
  }
  __syncthreads();
  const uint64_t b0 = (uint64_t)blockIdx.x * a.per_wave * kSortWaves;
  const uint64_t b1 = b0 + (uint64_t)a.per_wave * kSortWaves;
  const uint32_t end = (uint32_t)(b1 < a.n ? b1 : a.n);
  for (uint64_t j = b0 + threadIdx.x; j < end; j += kSortThreads) {
    const uint32_t key = FIRST ? key_of(a, (uint32_t)j) : a.from[j].key;
    atomicAdd(&hist[(key >> a.shift) & ((1u << a.bits) - 1u)], 1u);
  }
  __syncthreads();
  if (threadIdx.x < kBins) a.counts[blockIdx.x * kBins + threadIdx.x] = hist[threadIdx.x];
}

// Moves each token to its place: the tokens of smaller digits, then those of the same
// digit in earlier workgroups, earlier wavefronts and earlier in the wavefront.  Sixteen
// wavefronts a workgroup, for a wavefront's tokens go 64 at a time, one after another, and
// the workgroups' counts are added by four threads a pair of digits.
template <bool FIRST> __global__ __launch_bounds__(kSortThreads) void sort_scatter_kernel(SortArgs a) {
  constexpr uint32_t kPairs = kBins / 2, kShares = kSortThreads / kPairs;
  __shared__ uint32_t off[kSortWaves][kBins];
  __shared__ uint32_t total[kShares][kBins], before[kShares][kBins];
  __shared__ uint32_t wave_total[kSortWaves];
  const uint32_t t = threadIdx.x, wave = uniform(t / kWave), lane = lane_id();
  const uint64_t w0 = ((uint64_t)blockIdx.x * kSortWaves + wave) * a.per_wave;
  const uint64_t w1 = w0 + a.per_wave;
  const uint64_t end = w1 < a.n ? w1 : a.n;
  const uint32_t dm = (1u << a.bits) - 1u;
  auto load = [&](uint64_t j) {
    Pair p{0u, (uint32_t)j};
    if (j < end) {
      if constexpr (FIRST) p.key = key_of(a, (uint32_t)j);
      else p = a.from[j];
    }
    return p;
  };
  const Pair first = load(w0 + lane);
  {
    // tokens of each digit in all workgroups and in earlier ones, a share of the workgroups
    uint2 sum = make_uint2(0u, 0u), early = make_uint2(0u, 0u);
    const uint32_t pair = t % kPairs, share = t / kPairs;
    const uint2 *counts = reinterpret_cast<const uint2 *>(a.counts) + pair;
    constexpr uint32_t kFlight = 16;  // loads in flight: the counts come from L2
    for (uint32_t b0 = share; b0 < gridDim.x; b0 += kFlight * kShares) {
      uint2 v[kFlight];
#pragma unroll
      for (uint32_t k = 0; k < kFlight; ++k)
        v[k] = b0 + k * kShares < gridDim.x ? counts[(b0 + k * kShares) * kPairs] : make_uint2(0u, 0u);
#pragma unroll
      for (uint32_t k = 0; k < kFlight; ++k) {
        sum.x += v[k].x;
        sum.y += v[k].y;
        early.x += b0 + k * kShares < blockIdx.x ? v[k].x : 0u;
        early.y += b0 + k * kShares < blockIdx.x ? v[k].y : 0u;
      }
    }
    *reinterpret_cast<uint2 *>(&total[share][pair * 2]) = sum;
    *reinterpret_cast<uint2 *>(&before[share][pair * 2]) = early;
  }
  for (uint32_t i = t; i < kBins * kSortWaves; i += kSortThreads) (&off[0][0])[i] = 0;
  __syncthreads();
  if (w0 + lane < end) atomicAdd(&off[wave][(first.key >> a.shift) & dm], 1u);
  for (uint64_t j = w0 + kWave + lane; j < end; j += kWave) atomicAdd(&off[wave][(load(j).key >> a.shift) & dm], 1u);
  // thread d < kBins owns digit d
  uint32_t mine = 0, at = 0;
  if (t < kBins) {
#pragma unroll
    for (uint32_t k = 0; k < kShares; ++k) {
      mine += total[k][t];
      at += before[k][t];
    }
  }
  const uint32_t incl = wave_incl_scan(mine);
  if (lane == kWave - 1) wave_total[wave] = incl;
  __syncthreads();
  if (t < kBins) {
    at += incl - mine;
    for (uint32_t w = 0; w < wave; ++w) at += wave_total[w];
    uint32_t c[kSortWaves];
#pragma unroll
    for (uint32_t w = 0; w < kSortWaves; ++w) c[w] = off[w][t];
#pragma unroll
    for (uint32_t w = 0; w < kSortWaves; ++w) {
      off[w][t] = at;
      at += c[w];
    }
  }
  __syncthreads();
  for (uint64_t j0 = w0; j0 < end; j0 += kWave) {
    const bool live = j0 + lane < end;
    const Pair p = j0 == w0 ? first : load(j0 + lane);
    const uint32_t d = (p.key >> a.shift) & dm;
    const uint64_t same = same_digit(d, a.bits, ballot(live));
    const uint32_t rank = count_below(same);
    uint32_t to = 0;
    if (live) to = off[wave][d] + rank;
    wave_lds_sync();
    if (live && rank == 0) off[wave][d] += popc(same);
    wave_lds_sync();
    if (live && to < a.n) a.to[to] = p;  // always, unless the ids change while the call runs
  }
}

// The whole sort of up to kSmallTokens tokens in one workgroup, keys and positions in LDS.
// Further workgroups clear `clear` (n_clear elements) meanwhile.
template <int DO>
__global__ __launch_bounds__(kSortThreads) void sort_small_kernel(SortArgs a, uint32_t passes, uint32_t total_bits,
                                                                   void *clear, uint64_t n_clear) {
  if (blockIdx.x > 0) {
    using TO = typename Num<DO>::T;
    TO *p = static_cast<TO *>(clear);
    constexpr uint32_t kEach = 16 / sizeof(TO);
    typedef TO V __attribute__((ext_vector_type(kEach), aligned(sizeof(TO))));
    const uint64_t step = (uint64_t)(gridDim.x - 1) * kSortThreads * kEach;
    for (uint64_t i = ((uint64_t)(blockIdx.x - 1) * kSortThreads + threadIdx.x) * kEach; i < n_clear; i += step) {
      if (i + kEach <= n_clear) {
        *reinterpret_cast<V *>(p + i) = V{};
      } else {
        for (uint64_t e = i; e < n_clear; ++e) p[e] = (TO)0.0f;
      }
    }
    return;
  }
  __shared__ uint32_t keys[2][kSmallTokens];
  __shared__ uint16_t pos[2][kSmallTokens];
  static_assert(kSmallTokens <= 1u << 16, "positions in 16 bits");
  __shared__ uint32_t off[kSortWaves][kBins];
  __shared__ uint32_t wave_total[kSortWaves];
  const uint32_t t = threadIdx.x, wave = uniform(t / kWave), lane = lane_id();
  if (t == 0) a.crossing[0] = 0;
  for (uint32_t j = t; j < a.n; j += kSortThreads) {
    keys[0][j] = key_of(a, j);
    pos[0][j] = (uint16_t)j;
  }
  const uint32_t w0 = wave * a.per_wave, w1 = w0 + a.per_wave, end = w1 < a.n ? w1 : a.n;
  uint32_t shift = 0, cur = 0;
  for (uint32_t pass = 0; pass < passes; ++pass) {
    const uint32_t bits = total_bits - shift < a.bits ? total_bits - shift : a.bits, dm = (1u << bits) - 1u;
    for (uint32_t i = t; i < kBins * kSortWaves; i += kSortThreads) (&off[0][0])[i] = 0;
    __syncthreads();
    for (uint32_t j = w0 + lane; j < end; j += kWave) atomicAdd(&off[wave][(keys[cur][j] >> shift) & dm], 1u);
    __syncthreads();
    // thread d < kBins owns digit d
    uint32_t c[kSortWaves], mine = 0;
#pragma unroll
    for (uint32_t w = 0; w < kSortWaves; ++w) {
      c[w] = t < kBins ? off[w][t] : 0u;
      mine += c[w];
    }
    const uint32_t incl = wave_incl_scan(mine);
    if (lane == kWave - 1) wave_total[wave] = incl;
    __syncthreads();
    if (t < kBins) {
      uint32_t at = incl - mine;
      for (uint32_t w = 0; w < wave; ++w) at += wave_total[w];
#pragma unroll
      for (uint32_t w = 0; w < kSortWaves; ++w) {
        off[w][t] = at;
        at += c[w];
      }
    }
    __syncthreads();
    for (uint32_t j0 = w0; j0 < end; j0 += kWave) {
      const uint32_t j = j0 + lane;
      const bool live = j < end;
      const uint32_t key = live ? keys[cur][j] : 0u;
      const uint16_t at_j = live ? pos[cur][j] : 0;
      const uint32_t d = (key >> shift) & dm;
      const uint64_t same = same_digit(d, bits, ballot(live));
      const uint32_t rank = count_below(same);
      uint32_t at = 0;
      if (live) at = off[wave][d] + rank;
      wave_lds_sync();
      if (live && rank == 0) off[wave][d] += popc(same);
      wave_lds_sync();
      if (live) {
        keys[cur ^ 1][at] = key;
        pos[cur ^ 1][at] = at_j;
      }
    }
    __syncthreads();
    cur ^= 1;
    shift += bits;
  }
  for (uint32_t j = t; j < a.n; j += kSortThreads) a.to[j] = Pair{keys[cur][j], pos[cur][j]};
}

// ------------------------------------------------------------------ sums of the sorted rows

struct SumArgs {
  const void *dout;
  const Pair *sorted;
  void *grad;
  uint32_t *crossing;   // [0] how many chunks a run that is cut begins in, then those chunks in any order
  float *part;          // [chunk][2][dim]: sum of the chunk's first run when it began earlier, of its last when it goes on
  uint64_t n_rows;
  uint32_t n;
  uint32_t dim;
  uint32_t chunk;       // tokens per chunk
  uint32_t nchunks;
  uint32_t lanes;       // lanes a row, a power of two up to kBlock
  uint32_t slab;        // columns that a group of lanes covers: lanes * 8
  uint32_t slabs;       // ceil(dim / slab)
  uint32_t zero_blocks; // workgroups that write the rows without tokens; the rest sum
  float scale;
};

template <typename TO> __device__ __forceinline__ void put_row(const SumArgs &a, uint32_t row, uint32_t c, F8 v) {
#pragma unroll
  for (int i = 0; i < 8; ++i) v.v[i] *= a.scale;
  store8<TO>(static_cast<TO *>(a.grad) + (uint64_t)row * a.dim, c, a.dim, v);
}

// First of the sorted tokens [lo, hi) whose id is not below `key` (above it, with UPPER).
template <bool UPPER> __device__ __forceinline__ uint32_t bound(const Pair *sorted, uint32_t lo, uint32_t hi, uint32_t key) {
  while (lo < hi) {
    const uint32_t mid = lo + (hi - lo) / 2, k = sorted[mid].key;
    if (UPPER ? k <= key : k < key) lo = mid + 1;
    else hi = mid;
  }
  return lo;
}

// Sums columns [c, c + 8) of the rows of chunk ck: the runs that begin in it.  A run that
// fills no chunk is taken to its end, into the next chunk if need be; one that fills a
// chunk is cut at the chunks' borders, each chunk leaving a partial row.
template <bool WIDE, typename TI, typename TO> __device__ __forceinline__ void sum_chunk(const SumArgs &a, uint32_t ck, uint32_t c) {
  const TI *dout = static_cast<const TI *>(a.dout);
  const uint32_t i0 = ck * a.chunk, i1 = i0 + a.chunk < a.n ? i0 + a.chunk : a.n;
  const uint32_t none = (uint32_t)a.n_rows;
  uint32_t key = a.sorted[i0].key;
  const uint32_t last = a.sorted[i1 - 1].key;
  if (key == none) return;
  const bool full = key == last;
  const bool from_before = i0 > 0 && a.sorted[i0 - 1].key == key;
  bool first = from_before && (full || a.sorted[i0 - a.chunk].key == key);  // the rest of a run that is cut
  const bool goes_on = i1 < a.n && last != none && a.sorted[i1].key == last;
  const uint32_t i2 = i1 + a.chunk < a.n ? i1 + a.chunk : a.n;
  const bool cut = goes_on && (full || a.sorted[i2 - 1].key == last);
  const uint32_t begin = from_before && !first ? bound<true>(a.sorted, i0, i1, key) : i0;
  const uint32_t end = goes_on && !cut ? bound<true>(a.sorted, i1, i2, last) : i1;
  F8 acc{};
  float *part = a.part + (uint64_t)ck * 2 * a.dim;
  if (begin > i0) key = a.sorted[begin].key;  // not full: begin < i1
  constexpr uint32_t kFlight = 8;
  for (uint32_t i = begin; i < end; i += kFlight) {
    Pair p[kFlight];
    Vec8<TI> x[kFlight];
#pragma unroll
    for (uint32_t k = 0; k < kFlight; ++k) p[k] = a.sorted[i + k < end ? i + k : end - 1];
#pragma unroll
    for (uint32_t k = 0; k < kFlight; ++k) x[k] = load8<WIDE, TI>(dout + (uint64_t)p[k].pos * a.dim, c, a.dim);
#pragma unroll
    for (uint32_t k = 0; k < kFlight; ++k) {
      if (i + k >= end) break;
      if (p[k].key != key) {  // the run ended
        if (first) store8<float>(part, c, a.dim, acc);
        else if (key != none) put_row<TO>(a, key, c, acc);
        first = false;
        acc = F8{};
        key = p[k].key;
      }
      const F8 y = widen<WIDE, TI>(x[k], c, a.dim);
#pragma unroll
      for (int e = 0; e < 8; ++e) acc.v[e] += y.v[e];
    }
  }
  if (key == none) return;
  if (first) {
    store8<float>(part, c, a.dim, acc);
  } else if (cut) {
    store8<float>(part + a.dim, c, a.dim, acc);
    if (c == 0) a.crossing[1 + atomicAdd(a.crossing, 1u)] = ck;
  } else {
    put_row<TO>(a, key, c, acc);
  }
}

// zero_blocks workgroups write the rows without tokens, which they find by search in the
// sorted tokens, a lane a row; the others sum.
template <int DI, int DO> __global__ __launch_bounds__(kBlock) void grad_sum_kernel(SumArgs a) {
  using TI = typename Num<DI>::T;
  using TO = typename Num<DO>::T;
  const uint32_t tx = threadIdx.x & (a.lanes - 1), ty = threadIdx.x / a.lanes, groups = kBlock / a.lanes;
  // one of each in turn while there are both: reads and writes then share the memory
  const uint32_t sum_blocks = gridDim.x - a.zero_blocks, both = 2 * (sum_blocks < a.zero_blocks ? sum_blocks : a.zero_blocks);
  const bool zero = blockIdx.x < both ? blockIdx.x & 1 : sum_blocks < a.zero_blocks;
  const uint32_t block = blockIdx.x < both ? blockIdx.x >> 1 : blockIdx.x - both / 2;
  if (zero) {
    __shared__ uint64_t empty;
    for (uint64_t r0 = (uint64_t)block * kWave; r0 < a.n_rows; r0 += (uint64_t)a.zero_blocks * kWave) {
      if (threadIdx.x < kWave) {
        const uint64_t r = r0 + threadIdx.x;
        bool none = false;
        if (r < a.n_rows) {
          const uint32_t at = bound<false>(a.sorted, 0, a.n, (uint32_t)r);
          none = at >= a.n || a.sorted[at].key != (uint32_t)r;
        }
        const uint64_t m = ballot(none);
        if (threadIdx.x == 0) empty = m;
      }
      __syncthreads();
      const uint64_t m = empty;
      for (uint32_t k = ty; k < kWave; k += groups)
        if ((m >> k) & 1)
          for (uint32_t c = tx * 8; c < a.dim; c += a.slab)
            store8<TO>(static_cast<TO *>(a.grad) + (r0 + k) * a.dim, c, a.dim, F8{});
      __syncthreads();
    }
    return;
  }
  const uint64_t units = (uint64_t)a.nchunks * a.slabs, step = (uint64_t)sum_blocks * groups;
  by_width(a.dim, [&](auto wide) {
    for (uint64_t unit = (uint64_t)block * groups + ty; unit < units; unit += step) {
      const uint32_t c = (uint32_t)(unit % a.slabs) * a.slab + tx * 8;
      if (c < a.dim) sum_chunk<wide.value, TI, TO>(a, (uint32_t)(unit / a.slabs), c);
    }
  });
}

// Runs that are cut.  A workgroup takes a run and a strip of its columns; groups of
// lanes add consecutive shares of the run's partial rows (a frequent token has hundreds)
// and their sums are added in order, so the result does not depend on who took it.
template <int DO> __global__ __launch_bounds__(kBlock) void grad_join_kernel(SumArgs a, uint32_t lanes, uint32_t strips) {
  using TO = typename Num<DO>::T;
  __shared__ float sums[kBlock * 8];
  const uint32_t tx = threadIdx.x & (lanes - 1), ty = threadIdx.x / lanes, groups = kBlock / lanes;
  const uint64_t items = (uint64_t)a.crossing[0] * strips;
  by_width(a.dim, [&](auto wide) {
    for (uint64_t item = blockIdx.x; item < items; item += gridDim.x) {
      const uint32_t ck = a.crossing[1 + item / strips], c = ((uint32_t)(item % strips) * lanes + tx) * 8;
      const uint32_t key = a.sorted[(ck + 1) * a.chunk].key;
      uint32_t follow = 0, found;  // chunks after ck that begin with the run's id
      do {
        const uint32_t k = ck + 1 + follow + threadIdx.x;
        found = (uint32_t)__syncthreads_count(k < a.nchunks && a.sorted[k * a.chunk].key == key);
        follow += found;
      } while (found == kBlock);
      const uint32_t parts = follow + 1, share = (parts + groups - 1) / groups;
      const uint32_t p0 = ty * share, p1 = p0 + share < parts ? p0 + share : parts;
      // partial 0 is the last run of chunk ck, partial p the first of chunk ck + p
      auto row = [&](uint32_t p) { return a.part + ((uint64_t)(ck + p) * 2 + (p == 0)) * a.dim; };
      F8 acc{};
      constexpr uint32_t kFlight = 8;
      for (uint32_t p = p0; p < p1; p += kFlight) {
        Vec8<float> x[kFlight];
#pragma unroll
        for (uint32_t k = 0; k < kFlight; ++k) x[k] = load8<wide.value, float>(row(p + k < p1 ? p + k : p1 - 1), c, a.dim);
#pragma unroll
        for (uint32_t k = 0; k < kFlight; ++k)
          if (p + k < p1) {
            const F8 y = widen<wide.value, float>(x[k], c, a.dim);
#pragma unroll
            for (int e = 0; e < 8; ++e) acc.v[e] += y.v[e];
          }
      }
#pragma unroll
      for (int e = 0; e < 8; ++e) sums[e * kBlock + threadIdx.x] = acc.v[e];
      __syncthreads();
      if (ty == 0 && c < a.dim) {
        for (uint32_t g = 1; g < groups && g * share < parts; ++g) {
#pragma unroll
          for (int e = 0; e < 8; ++e) acc.v[e] += sums[e * kBlock + g * lanes + tx];
        }
        put_row<TO>(a, key, c, acc);
      }
      __syncthreads();
    }
  });
}

// ------------------------------------------------------------------ host side

// Tokens per chunk.  Where the elements are few, short chunks: a group of lanes takes a
// chunk's tokens one after another, and more groups work.  Where they or the tokens are many,
// long ones: each chunk may leave two 32-bit partial rows.  Chunks of 4, 8, 16 and 32, frequent
// ids: 7744 tokens of 21 30.1, 32.2, 38.5, 49.6 us; 8192 of 256 33.5, 31.8, 33.8, 39.0; 65536
// of 64 55.2, 46.5, 43.8, 46.5; 16384 of 1024 75.2, 67.3, 62.5, 53.7; 1000000 of 64 356, 219,
// 173, 144.  A few tokens are one chunk, so that no run is cut and no second kernel needed
// (16 of 64: 13.0 us of host and kernels against 16.4; 32 of 4096 17.0 against 16.5).
uint32_t grad_chunk(uint64_t n, uint32_t dim) {
  const uint64_t elements = n * dim;
  if (n <= 16) return 16;
  if (elements >= 1u << 24 || n >= 131072) return 32;
  if (elements >= 1u << 23 || n >= 65536) return 16;
  return elements >= 1u << 20 || n >= 16384 ? 8 : 4;
}

uint64_t up16(uint64_t v) { return (v + 15) & ~15ull; }

struct GradLayout {
  uint64_t pairs, counts, crossing, part, bytes;  // byte offsets: two pair lists at pairs
};

GradLayout grad_layout(uint64_t n, uint32_t dim) {
  GradLayout l;
  l.pairs = 0;
  l.counts = up16(2 * n * sizeof(Pair));
  l.crossing = l.counts + kSortBlocks * kBins * 4;
  const uint64_t ck = grad_chunk(n, dim), chunks = (n + ck - 1) / ck;
  l.part = l.crossing + up16(4 * (chunks + 1));
  l.bytes = l.part + chunks * 2 * dim * 4;
  return l;
}

}  // namespace

uint64_t embed_grad_workspace(uint64_t, uint64_t n_ids, uint32_t dim) {
  return grad_layout(n_ids, dim).bytes;
}

hipError_t launch_lookup(const LookupArgs &a, hipStream_t s) {
  RowWalk w;
  w.lanes = pow2_lanes(a.dim);
  // Four rows a lane, and all their columns by one workgroup, where that leaves the GPU
  // full; else a row each, its columns shared out, so that few tokens spread over the CUs (bf16,
  // four rows against one; 512 columns: 4096 tokens 3.9 us and 3.5, 8192 4.7 and 4.8, 16384 6.7
  // and 7.2; 4096 columns: 512 tokens 4.9 and 3.6, 4096 12.8 and 12.5, 16384 44 and 52).
  const uint64_t four_rows = (uint64_t)(kBlock / w.lanes) * 4, fours = (a.n_ids + four_rows - 1) / four_rows;
  const bool four = fours >= 1024;
  const uint64_t one_rows = kBlock / w.lanes;
  w.strips = four ? 1 : ((a.dim + 7) / 8 + w.lanes - 1) / w.lanes;
  w.units = four ? fours : (a.n_ids + one_rows - 1) / one_rows * w.strips;
  const uint32_t blocks = (uint32_t)(w.units < (1u << 22) ? w.units : (1u << 22));
  return with_dtype(a.in_dtype, [&](auto di) {
    return with_dtype(a.out_dtype, [&](auto dO) {
      if (four) lookup_kernel<di.value, dO.value, 4><<<blocks, kBlock, 0, s>>>(a, w);
      else lookup_kernel<di.value, dO.value, 1><<<blocks, kBlock, 0, s>>>(a, w);
      return hipGetLastError();
    });
  });
}

hipError_t launch_embed_grad(const EmbedGradArgs &a, hipStream_t s) {
  const GradLayout l = grad_layout(a.n_ids, a.dim);
  Pair *pa = reinterpret_cast<Pair *>(a.ws + l.pairs), *pb = pa + a.n_ids;
  SortArgs so;
  so.ids = a.ids;
  so.err = a.err;
  so.from = pb;
  so.to = pa;
  so.counts = reinterpret_cast<uint32_t *>(a.ws + l.counts);
  so.crossing = reinterpret_cast<uint32_t *>(a.ws + l.crossing);
  so.n_rows = a.n_rows;
  so.padding_id = a.padding_id;
  so.n = (uint32_t)a.n_ids;
  const uint32_t total_bits = 64u - (uint32_t)__builtin_clzll(a.n_rows);  // keys 0..n_rows
  const uint32_t passes = (total_bits + kDigitBits - 1) / kDigitBits;
  so.bits = (total_bits + passes - 1) / passes;
  so.shift = 0;
  // One workgroup can sort up to kSmallTokens while others clear every row: that writes the
  // tokens' rows twice, but takes one kernel and hides the sort.  Else the summing kernel
  // clears the rows without tokens.  4000 tokens of 1000, frequent ids, 16000 rows: 28 us, with
  // this sort and clearing by sums 42, with many workgroups' sort 47; 4000 rows: 26, 29, 33.
  // Above 4096 tokens one workgroup sorts slower than many, so there has to be enough to
  // clear: 8192 tokens of 4096, 8000 rows (131 MB): 70 us against 84 by many, of 1000, 8000
  // rows (32 MB): 40 against 40, of 64, 32000 rows (8 MB): 40 against 36.
  const uint64_t grad_bytes = a.n_rows * a.dim * (a.out_dtype == IBP_F32 ? 4 : 2);
  const bool clear_first = a.n_ids <= 4096 || (a.n_ids <= kSmallTokens && grad_bytes >= 32u << 20);
  hipError_t e = hipSuccess;
  const Pair *sorted = pa;
  if (clear_first) {
    const uint32_t per = (so.n + kSortThreads - 1) / kSortThreads;
    so.per_wave = (per ? per : 1) * kWave;
    const uint64_t want = (a.n_rows * a.dim + kSortThreads * 8 - 1) / (kSortThreads * 8);
    const uint32_t clearers = (uint32_t)(want < 512 ? want : 512);
    e = with_dtype(a.out_dtype, [&](auto d) {
      sort_small_kernel<d.value><<<1 + clearers, kSortThreads, 0, s>>>(so, passes, total_bits, a.grad, a.n_rows * a.dim);
      return hipGetLastError();
    });
  } else {
    const uint64_t want = (a.n_ids + kSortMin - 1) / kSortMin;
    const uint32_t blocks = (uint32_t)(want < kSortBlocks ? want : kSortBlocks);
    const uint64_t per = (a.n_ids + (uint64_t)blocks * kSortThreads - 1) / ((uint64_t)blocks * kSortThreads);
    so.per_wave = (uint32_t)per * kWave;
    for (uint32_t p = 0; p < passes && e == hipSuccess; ++p) {
      SortArgs q = so;
      q.shift = p * so.bits;
      q.bits = total_bits - q.shift < so.bits ? total_bits - q.shift : so.bits;
      q.to = p & 1 ? pb : pa;
      q.from = p & 1 ? pa : pb;
      if (p == 0) sort_count_kernel<true><<<blocks, kSortThreads, 0, s>>>(q);
      else sort_count_kernel<false><<<blocks, kSortThreads, 0, s>>>(q);
      e = hipGetLastError();
      if (e != hipSuccess) break;
      if (p == 0) sort_scatter_kernel<true><<<blocks, kSortThreads, 0, s>>>(q);
      else sort_scatter_kernel<false><<<blocks, kSortThreads, 0, s>>>(q);
      e = hipGetLastError();
      sorted = q.to;
    }
  }
  if (e != hipSuccess) return e;
  SumArgs m;
  m.dout = a.dout;
  m.sorted = sorted;
  m.grad = a.grad;
  m.crossing = so.crossing;
  m.part = reinterpret_cast<float *>(a.ws + l.part);
  m.n_rows = a.n_rows;
  m.n = so.n;
  m.dim = a.dim;
  m.chunk = grad_chunk(a.n_ids, a.dim);
  m.nchunks = (m.n + m.chunk - 1) / m.chunk;
  m.lanes = pow2_lanes(a.dim);
  m.slab = m.lanes * 8;
  m.slabs = (a.dim + m.slab - 1) / m.slab;
  m.scale = a.scale;
  const uint32_t groups = kBlock / m.lanes;
  uint64_t sum_blocks = ((uint64_t)m.nchunks * m.slabs + groups - 1) / groups;
  if (sum_blocks > (1u << 22)) sum_blocks = 1u << 22;
  const uint64_t zero = (a.n_rows + kWave - 1) / kWave;
  const uint64_t zero_blocks = clear_first ? 0 : zero < 8192 ? zero : 8192;
  m.zero_blocks = (uint32_t)zero_blocks;
  if (sum_blocks + zero_blocks == 0) return e;  // no tokens, rows cleared
  e = with_dtype(a.in_dtype, [&](auto di) {
    return with_dtype(a.out_dtype, [&](auto dO) {
      grad_sum_kernel<di.value, dO.value><<<(uint32_t)(sum_blocks + zero_blocks), kBlock, 0, s>>>(m);
      return hipGetLastError();
    });
  });
  if (e != hipSuccess || m.nchunks < 2) return e;
  const uint32_t lanes = m.lanes < 32 ? m.lanes : 32, strips = (a.dim + lanes * 8 - 1) / (lanes * 8);
  const uint64_t items = (uint64_t)m.nchunks * strips;  // at most
  return with_dtype(a.out_dtype, [&](auto dO) {
    grad_join_kernel<dO.value><<<(uint32_t)(items < 1024 ? items : 1024), kBlock, 0, s>>>(m, lanes, strips);
    return hipGetLastError();
  });
}

}  // namespace ibp
