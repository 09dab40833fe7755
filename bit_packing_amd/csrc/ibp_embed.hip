// ibp_embed.hip -- embedding lookup with scaling, and its gradient by sorted tokens.
//
// Lookup: out[j] = scale * table[ids[j]], one read of each token's row and one write.
// Bound by HBM; a lane moves eight elements, a row is taken by the smallest power of
// two of lanes that covers it, and a lane has kRowsEach rows in flight.
//
// Gradient: grad[v] = scale * sum of dout[j] over the tokens j with ids[j] == v, in
// 32 bits, rows without tokens 0.  Tokens are sorted by id (stable, so a row's tokens
// keep their order and the sums do not depend on timing), the sorted list is cut into
// chunks of equal length, and each chunk's rows are summed by one group of lanes: the
// work is even however unevenly the tokens fall on the rows.  A run of equal ids that
// lies inside a chunk is finished there; a run that crosses chunks leaves one 32-bit
// partial row per chunk, and a second kernel adds those in order.  dout is read once
// and grad written once; the sort moves 8 bytes a token a pass.
#include "ibp_device.h"
#include "ibp_num.h"

namespace ibp {
namespace {

using namespace dev;

// ------------------------------------------------------------------ lookup

constexpr uint32_t kRowsEach = 4;

struct RowWalk {
  uint32_t lanes;     // lanes a row, a power of two up to kBlock
  uint32_t rows_blk;  // kBlock / lanes
  uint64_t steps;
};

uint32_t pow2_lanes(uint32_t dim) {
  uint32_t l = 1;
  while (l < (dim + 7) / 8 && l < kBlock) l *= 2;
  return l;
}

template <int DI, int DO> __global__ __launch_bounds__(kBlock) void lookup_kernel(LookupArgs a, RowWalk w) {
  using TI = typename Num<DI>::T;
  using TO = typename Num<DO>::T;
  const uint32_t tx = threadIdx.x & (w.lanes - 1), ty = threadIdx.x / w.lanes;
  const TI *table = static_cast<const TI *>(a.table);
  TO *out = static_cast<TO *>(a.out);
  for (uint64_t step = blockIdx.x; step < w.steps; step += gridDim.x) {
    const uint64_t j0 = step * w.rows_blk * kRowsEach + ty;
    uint64_t id[kRowsEach];
    bool ok[kRowsEach], live[kRowsEach];
#pragma unroll
    for (uint32_t k = 0; k < kRowsEach; ++k) {
      const uint64_t j = j0 + (uint64_t)k * w.rows_blk;
      live[k] = j < a.n_ids;
      const int64_t v = live[k] ? a.ids[j] : -1;
      ok[k] = v >= 0 && (uint64_t)v < a.n_rows;
      id[k] = ok[k] ? (uint64_t)v : 0;
      if (live[k] && !ok[k] && tx == 0 && a.err) atomicOr(a.err, IBP_DEVERR_BAD_ID);
    }
    for (uint32_t c = tx * 8; c < a.dim; c += w.lanes * 8) {
      Vec8<TI> x[kRowsEach];
#pragma unroll
      for (uint32_t k = 0; k < kRowsEach; ++k) x[k] = load8<TI>(table + id[k] * a.dim, c, a.dim);
#pragma unroll
      for (uint32_t k = 0; k < kRowsEach; ++k) {
        if (!live[k]) continue;
        F8 y = widen<TI>(x[k]);
#pragma unroll
        for (int i = 0; i < 8; ++i) y.v[i] = ok[k] ? y.v[i] * a.scale : 0.0f;
        store8<TO>(out + (j0 + (uint64_t)k * w.rows_blk) * a.dim, c, a.dim, y);
      }
    }
  }
}

// ------------------------------------------------------------------ sort by id

// Radix sort of (key, position) pairs, keys 0..n_rows; key n_rows stands for tokens
// that take no part (the padding id, ids out of range) and sorts to the end.  Digits
// of up to nine bits: two passes cover 2^18 rows.
constexpr uint32_t kDigitBits = 9, kBins = 1u << kDigitBits;
constexpr uint32_t kSortBlocks = 256;     // at most this many workgroups a pass
constexpr uint32_t kSortMin = 1024;       // tokens per workgroup at least
constexpr uint32_t kSmallTokens = 4096;   // sorted by one workgroup in LDS
constexpr uint32_t kSmallThreads = 1024;

struct Pair { uint32_t key, pos; };

struct SortArgs {
  const int64_t *ids;
  uint32_t *err;
  Pair *from, *to;      // from: unused by the first pass
  uint32_t *counts;     // [workgroup][kBins]
  uint32_t *present;    // bit per row: has tokens
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

__device__ __forceinline__ void mark_present(uint32_t *present, uint32_t key) {
  const uint32_t bit = 1u << (key & 31);
  if (!(__hip_atomic_load(&present[key >> 5], __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT) & bit))
    atomicOr(&present[key >> 5], bit);
}

// Per workgroup, how many of its tokens have each digit.  The first pass also clears
// the presence bits that the next kernel sets.
template <bool FIRST> __global__ __launch_bounds__(kBlock) void sort_count_kernel(SortArgs a) {
  __shared__ uint32_t hist[kBins];
  for (uint32_t i = threadIdx.x; i < kBins; i += kBlock) hist[i] = 0;
  if constexpr (FIRST) {
    const uint64_t words = (a.n_rows + 31) / 32;
    for (uint64_t i = (uint64_t)blockIdx.x * kBlock + threadIdx.x; i < words; i += (uint64_t)gridDim.x * kBlock)
      a.present[i] = 0;
  }
  __syncthreads();
  const uint64_t b0 = (uint64_t)blockIdx.x * a.per_wave * kWavesPerBlock;
  const uint64_t b1 = b0 + (uint64_t)a.per_wave * kWavesPerBlock;
  const uint32_t end = (uint32_t)(b1 < a.n ? b1 : a.n);
  for (uint64_t j = b0 + threadIdx.x; j < end; j += kBlock) {
    const uint32_t key = FIRST ? key_of(a, (uint32_t)j) : a.from[j].key;
    atomicAdd(&hist[(key >> a.shift) & ((1u << a.bits) - 1u)], 1u);
  }
  __syncthreads();
  for (uint32_t i = threadIdx.x; i < kBins; i += kBlock) a.counts[blockIdx.x * kBins + i] = hist[i];
}

// Moves each token to its place: the tokens of smaller digits, then those of the same
// digit in earlier workgroups, earlier wavefronts and earlier in the wavefront.
template <bool FIRST> __global__ __launch_bounds__(kBlock) void sort_scatter_kernel(SortArgs a) {
  __shared__ uint32_t off[kWavesPerBlock][kBins];
  __shared__ uint32_t wave_total[kWavesPerBlock];
  const uint32_t wave = uniform(threadIdx.x / kWave), lane = lane_id();
  for (uint32_t i = threadIdx.x; i < kBins * kWavesPerBlock; i += kBlock) (&off[0][0])[i] = 0;
  __syncthreads();
  const uint64_t w0 = ((uint64_t)blockIdx.x * kWavesPerBlock + wave) * a.per_wave;
  const uint64_t w1 = w0 + a.per_wave;
  const uint64_t end = w1 < a.n ? w1 : a.n;
  const uint32_t dm = (1u << a.bits) - 1u;
  for (uint64_t j = w0 + lane; j < end; j += kWave) {
    const uint32_t key = FIRST ? key_of(a, (uint32_t)j) : a.from[j].key;
    atomicAdd(&off[wave][(key >> a.shift) & dm], 1u);
  }
  // totals of each digit, and its tokens in earlier workgroups; two digits a thread
  constexpr uint32_t kEach = kBins / kBlock;
  uint32_t total[kEach] = {}, before[kEach] = {};
  for (uint32_t b = 0; b < gridDim.x; ++b) {
#pragma unroll
    for (uint32_t e = 0; e < kEach; ++e) {
      const uint32_t v = a.counts[b * kBins + threadIdx.x * kEach + e];
      total[e] += v;
      before[e] += b < blockIdx.x ? v : 0u;
    }
  }
  uint32_t mine = 0;
#pragma unroll
  for (uint32_t e = 0; e < kEach; ++e) mine += total[e];
  const uint32_t incl = wave_incl_scan(mine);
  if (lane == kWave - 1) wave_total[wave] = incl;
  __syncthreads();
  uint32_t base = incl - mine;
  for (uint32_t w = 0; w < wave; ++w) base += wave_total[w];
#pragma unroll
  for (uint32_t e = 0; e < kEach; ++e) {
    uint32_t at = base + before[e];
    base += total[e];
    for (uint32_t w = 0; w < kWavesPerBlock; ++w) {
      const uint32_t c = off[w][threadIdx.x * kEach + e];
      off[w][threadIdx.x * kEach + e] = at;
      at += c;
    }
  }
  __syncthreads();
  for (uint64_t j0 = w0; j0 < end; j0 += kWave) {
    const uint64_t j = j0 + lane;
    const bool live = j < end;
    Pair p{0u, (uint32_t)j};
    if (live) {
      if constexpr (FIRST) p.key = key_of(a, (uint32_t)j);
      else p = a.from[j];
    }
    const uint32_t d = (p.key >> a.shift) & dm;
    const uint64_t same = same_digit(d, a.bits, ballot(live));
    const uint32_t rank = count_below(same);
    uint32_t at = 0;
    if (live) at = off[wave][d] + rank;
    wave_lds_sync();
    if (live && rank == 0) off[wave][d] += popc(same);
    wave_lds_sync();
    if (live && at < a.n) {  // always, unless the ids change while the call runs
      a.to[at] = p;
      if (FIRST && p.key < a.n_rows) mark_present(a.present, p.key);
    }
  }
}

// The whole sort of up to kSmallTokens tokens in one workgroup, pairs in LDS.
__global__ __launch_bounds__(kSmallThreads) void sort_small_kernel(SortArgs a, uint32_t passes, uint32_t total_bits) {
  constexpr uint32_t kWaves = kSmallThreads / kWave;
  __shared__ Pair buf[2][kSmallTokens];
  __shared__ uint32_t off[kWaves][kBins];
  __shared__ uint32_t wave_total[kWaves];
  const uint32_t t = threadIdx.x, wave = uniform(t / kWave), lane = lane_id();
  const uint64_t words = (a.n_rows + 31) / 32;
  for (uint64_t i = t; i < words; i += kSmallThreads) a.present[i] = 0;
  __threadfence();  // before other wavefronts set bits of them
  for (uint32_t j = t; j < a.n; j += kSmallThreads) buf[0][j] = Pair{key_of(a, j), j};
  const uint32_t w0 = wave * a.per_wave, w1 = w0 + a.per_wave, end = w1 < a.n ? w1 : a.n;
  uint32_t shift = 0, cur = 0;
  for (uint32_t pass = 0; pass < passes; ++pass) {
    const uint32_t bits = total_bits - shift < a.bits ? total_bits - shift : a.bits, dm = (1u << bits) - 1u;
    for (uint32_t i = t; i < kBins * kWaves; i += kSmallThreads) (&off[0][0])[i] = 0;
    __syncthreads();
    for (uint32_t j = w0 + lane; j < end; j += kWave) atomicAdd(&off[wave][(buf[cur][j].key >> shift) & dm], 1u);
    __syncthreads();
    // thread d < kBins owns digit d
    uint32_t mine = 0;
    if (t < kBins)
      for (uint32_t w = 0; w < kWaves; ++w) mine += off[w][t];
    const uint32_t incl = wave_incl_scan(mine);
    if (lane == kWave - 1) wave_total[wave] = incl;
    __syncthreads();
    if (t < kBins) {
      uint32_t at = incl - mine;
      for (uint32_t w = 0; w < wave; ++w) at += wave_total[w];
      for (uint32_t w = 0; w < kWaves; ++w) {
        const uint32_t c = off[w][t];
        off[w][t] = at;
        at += c;
      }
    }
    __syncthreads();
    for (uint32_t j0 = w0; j0 < end; j0 += kWave) {
      const uint32_t j = j0 + lane;
      const bool live = j < end;
      const Pair p = live ? buf[cur][j] : Pair{0u, 0u};
      const uint32_t d = (p.key >> shift) & dm;
      const uint64_t same = same_digit(d, bits, ballot(live));
      const uint32_t rank = count_below(same);
      uint32_t at = 0;
      if (live) at = off[wave][d] + rank;
      wave_lds_sync();
      if (live && rank == 0) off[wave][d] += popc(same);
      wave_lds_sync();
      if (live) buf[cur ^ 1][at] = p;
    }
    __syncthreads();
    cur ^= 1;
    shift += bits;
  }
  for (uint32_t j = t; j < a.n; j += kSmallThreads) {
    const Pair p = buf[cur][j];
    a.to[j] = p;
    if (p.key < a.n_rows) mark_present(a.present, p.key);
  }
}

// ------------------------------------------------------------------ sums of the sorted rows

struct SumArgs {
  const void *dout;
  const Pair *sorted;
  const uint32_t *present;
  void *grad;
  float *part;          // [chunk][2][dim]: sum of the chunk's first run when it began earlier, of its last when it goes on
  uint64_t n_rows;
  uint32_t n;
  uint32_t dim;
  uint32_t chunk;       // tokens per chunk
  uint32_t nchunks;
  uint32_t lanes;       // lanes a row, a power of two up to kBlock
  uint32_t slab;        // columns that a group of lanes covers: lanes * 8
  uint32_t slabs;       // ceil(dim / slab)
  uint32_t sum_blocks;  // workgroups that sum; the rest write zeros
  float scale;
};

template <typename TO> __device__ __forceinline__ void put_row(const SumArgs &a, uint32_t row, uint32_t c, F8 v) {
#pragma unroll
  for (int i = 0; i < 8; ++i) v.v[i] *= a.scale;
  store8<TO>(static_cast<TO *>(a.grad) + (uint64_t)row * a.dim, c, a.dim, v);
}

// Sums columns [c, c + 8) of the rows of chunk ck.
template <typename TI, typename TO> __device__ __forceinline__ void sum_chunk(const SumArgs &a, uint32_t ck, uint32_t c) {
  const TI *dout = static_cast<const TI *>(a.dout);
  const uint32_t i0 = ck * a.chunk, i1 = i0 + a.chunk < a.n ? i0 + a.chunk : a.n;
  const uint32_t none = (uint32_t)a.n_rows;
  uint32_t key = a.sorted[i0].key;
  if (key == none) return;
  bool first = i0 > 0 && a.sorted[i0 - 1].key == key;  // the run began in an earlier chunk
  F8 acc{};
  float *part = a.part + (uint64_t)ck * 2 * a.dim;
  constexpr uint32_t kFlight = 8;
  for (uint32_t i = i0; i < i1; i += kFlight) {
    Pair p[kFlight];
    Vec8<TI> x[kFlight];
#pragma unroll
    for (uint32_t k = 0; k < kFlight; ++k) p[k] = a.sorted[i + k < i1 ? i + k : i1 - 1];
#pragma unroll
    for (uint32_t k = 0; k < kFlight; ++k) x[k] = load8<TI>(dout + (uint64_t)p[k].pos * a.dim, c, a.dim);
#pragma unroll
    for (uint32_t k = 0; k < kFlight; ++k) {
      if (i + k >= i1) break;
      if (p[k].key != key) {  // the run ended inside the chunk
        if (first) store8<float>(part, c, a.dim, acc);
        else if (key != none) put_row<TO>(a, key, c, acc);
        first = false;
        acc = F8{};
        key = p[k].key;
      }
      const F8 y = widen<TI>(x[k]);
#pragma unroll
      for (int e = 0; e < 8; ++e) acc.v[e] += y.v[e];
    }
  }
  if (key == none) return;
  if (first) store8<float>(part, c, a.dim, acc);
  else if (i1 < a.n && a.sorted[i1].key == key) store8<float>(part + a.dim, c, a.dim, acc);
  else put_row<TO>(a, key, c, acc);
}

template <int DI, int DO> __global__ __launch_bounds__(kBlock) void grad_sum_kernel(SumArgs a) {
  using TI = typename Num<DI>::T;
  using TO = typename Num<DO>::T;
  const uint32_t tx = threadIdx.x & (a.lanes - 1), ty = threadIdx.x / a.lanes, groups = kBlock / a.lanes;
  if (blockIdx.x >= a.sum_blocks) {
    // rows without tokens are 0
    const uint32_t zb = blockIdx.x - a.sum_blocks, zn = gridDim.x - a.sum_blocks;
    for (uint64_t r = (uint64_t)zb * groups + ty; r < a.n_rows; r += (uint64_t)zn * groups)
      if (!((a.present[r >> 5] >> (r & 31)) & 1u))
        for (uint32_t c = tx * 8; c < a.dim; c += a.slab)
          store8<TO>(static_cast<TO *>(a.grad) + r * a.dim, c, a.dim, F8{});
    return;
  }
  const uint64_t units = (uint64_t)a.nchunks * a.slabs;
  for (uint64_t unit = (uint64_t)blockIdx.x * groups + ty; unit < units; unit += (uint64_t)a.sum_blocks * groups) {
    const uint32_t c = (uint32_t)(unit % a.slabs) * a.slab + tx * 8;
    if (c < a.dim) sum_chunk<TI, TO>(a, (uint32_t)(unit / a.slabs), c);
  }
}

// Runs that cross chunks: the group of the chunk in which such a run begins adds its
// partial rows in order.
template <typename TO> __device__ __forceinline__ void join_chunk(const SumArgs &a, uint32_t ck, uint32_t c) {
  const uint32_t i0 = ck * a.chunk, i1 = i0 + a.chunk;
  if (i1 >= a.n) return;
  const uint32_t key = a.sorted[i1 - 1].key;
  if (key == (uint32_t)a.n_rows || a.sorted[i1].key != key) return;
  if (i0 > 0 && a.sorted[i0 - 1].key == key) return;  // sorted: it then fills this chunk and began earlier
  uint32_t lo = i1 + 1, hi = a.n;  // first token after the run
  while (lo < hi) {
    const uint32_t mid = lo + (hi - lo) / 2;
    if (a.sorted[mid].key == key) lo = mid + 1;
    else hi = mid;
  }
  const uint32_t last = (lo - 1) / a.chunk;
  F8 acc = widen<float>(load8<float>(a.part + ((uint64_t)ck * 2 + 1) * a.dim, c, a.dim));
  constexpr uint32_t kFlight = 8;
  for (uint32_t k0 = ck + 1; k0 <= last; k0 += kFlight) {
    Vec8<float> x[kFlight];
#pragma unroll
    for (uint32_t k = 0; k < kFlight; ++k)
      x[k] = load8<float>(a.part + (uint64_t)(k0 + k <= last ? k0 + k : last) * 2 * a.dim, c, a.dim);
#pragma unroll
    for (uint32_t k = 0; k < kFlight; ++k)
      if (k0 + k <= last) {
#pragma unroll
        for (int e = 0; e < 8; ++e) acc.v[e] += x[k][e];
      }
  }
  put_row<TO>(a, key, c, acc);
}

template <int DO> __global__ __launch_bounds__(kBlock) void grad_join_kernel(SumArgs a) {
  using TO = typename Num<DO>::T;
  const uint32_t tx = threadIdx.x & (a.lanes - 1), ty = threadIdx.x / a.lanes, groups = kBlock / a.lanes;
  const uint64_t units = (uint64_t)a.nchunks * a.slabs;
  for (uint64_t unit = (uint64_t)blockIdx.x * groups + ty; unit < units; unit += (uint64_t)gridDim.x * groups) {
    const uint32_t c = (uint32_t)(unit % a.slabs) * a.slab + tx * 8;
    if (c < a.dim) join_chunk<TO>(a, (uint32_t)(unit / a.slabs), c);
  }
}

// ------------------------------------------------------------------ host side

// Tokens per chunk: short sequences take short chunks, or too few groups would work;
// long ones amortise the partial rows (two 32-bit rows a chunk at most).
uint32_t grad_chunk(uint64_t n) { return n < 32768 ? 8 : 32; }

uint64_t up16(uint64_t v) { return (v + 15) & ~15ull; }

struct GradLayout {
  uint64_t pairs, counts, present, part, bytes;  // byte offsets: two pair lists at pairs
};

GradLayout grad_layout(uint64_t n_rows, uint64_t n, uint32_t dim) {
  GradLayout l;
  l.pairs = 0;
  l.counts = up16(2 * n * sizeof(Pair));
  l.present = l.counts + kSortBlocks * kBins * 4;
  l.part = l.present + up16((n_rows + 31) / 32 * 4);
  const uint32_t ck = grad_chunk(n);
  l.bytes = l.part + (n + ck - 1) / ck * 2 * dim * 4ull;
  return l;
}

}  // namespace

uint64_t embed_grad_workspace(uint64_t n_rows, uint64_t n_ids, uint32_t dim) {
  return grad_layout(n_rows, n_ids, dim).bytes;
}

hipError_t launch_lookup(const LookupArgs &a, hipStream_t s) {
  RowWalk w;
  w.lanes = pow2_lanes(a.dim);
  w.rows_blk = kBlock / w.lanes;
  const uint64_t each = (uint64_t)w.rows_blk * kRowsEach;
  w.steps = (a.n_ids + each - 1) / each;
  const uint32_t blocks = (uint32_t)(w.steps < (1u << 22) ? w.steps : (1u << 22));
  return with_dtype(a.in_dtype, [&](auto di) {
    return with_dtype(a.out_dtype, [&](auto dO) {
      lookup_kernel<di.value, dO.value><<<blocks, kBlock, 0, s>>>(a, w);
      return hipGetLastError();
    });
  });
}

hipError_t launch_embed_grad(const EmbedGradArgs &a, hipStream_t s) {
  const GradLayout l = grad_layout(a.n_rows, a.n_ids, a.dim);
  Pair *pa = reinterpret_cast<Pair *>(a.ws + l.pairs), *pb = pa + a.n_ids;
  SortArgs so;
  so.ids = a.ids;
  so.err = a.err;
  so.from = pb;
  so.to = pa;
  so.counts = reinterpret_cast<uint32_t *>(a.ws + l.counts);
  so.present = reinterpret_cast<uint32_t *>(a.ws + l.present);
  so.n_rows = a.n_rows;
  so.padding_id = a.padding_id;
  so.n = (uint32_t)a.n_ids;
  const uint32_t total_bits = 64u - (uint32_t)__builtin_clzll(a.n_rows);  // keys 0..n_rows
  const uint32_t passes = (total_bits + kDigitBits - 1) / kDigitBits;
  so.bits = (total_bits + passes - 1) / passes;
  so.shift = 0;
  hipError_t e = hipSuccess;
  const Pair *sorted = pa;
  if (a.n_ids <= kSmallTokens) {
    const uint32_t per = (so.n + kSmallThreads - 1) / kSmallThreads;
    so.per_wave = (per ? per : 1) * kWave;
    sort_small_kernel<<<1, kSmallThreads, 0, s>>>(so, passes, total_bits);
    e = hipGetLastError();
  } else {
    const uint64_t want = (a.n_ids + kSortMin - 1) / kSortMin;
    const uint32_t blocks = (uint32_t)(want < kSortBlocks ? want : kSortBlocks);
    const uint64_t per = (a.n_ids + (uint64_t)blocks * kBlock - 1) / ((uint64_t)blocks * kBlock);
    so.per_wave = (uint32_t)per * kWave;
    for (uint32_t p = 0; p < passes && e == hipSuccess; ++p) {
      SortArgs q = so;
      q.shift = p * so.bits;
      q.bits = total_bits - q.shift < so.bits ? total_bits - q.shift : so.bits;
      q.to = p & 1 ? pb : pa;
      q.from = p & 1 ? pa : pb;
      if (p == 0) sort_count_kernel<true><<<blocks, kBlock, 0, s>>>(q);
      else sort_count_kernel<false><<<blocks, kBlock, 0, s>>>(q);
      e = hipGetLastError();
      if (e != hipSuccess) break;
      if (p == 0) sort_scatter_kernel<true><<<blocks, kBlock, 0, s>>>(q);
      else sort_scatter_kernel<false><<<blocks, kBlock, 0, s>>>(q);
      e = hipGetLastError();
      sorted = q.to;
    }
  }
  if (e != hipSuccess) return e;
  SumArgs m;
  m.dout = a.dout;
  m.sorted = sorted;
  m.present = so.present;
  m.grad = a.grad;
  m.part = reinterpret_cast<float *>(a.ws + l.part);
  m.n_rows = a.n_rows;
  m.n = so.n;
  m.dim = a.dim;
  m.chunk = grad_chunk(a.n_ids);
  m.nchunks = (m.n + m.chunk - 1) / m.chunk;
  m.lanes = pow2_lanes(a.dim);
  m.slab = m.lanes * 8;
  m.slabs = (a.dim + m.slab - 1) / m.slab;
  m.scale = a.scale;
  const uint32_t groups = kBlock / m.lanes;
  uint64_t sum_blocks = ((uint64_t)m.nchunks * m.slabs + groups - 1) / groups;
  if (sum_blocks > (1u << 22)) sum_blocks = 1u << 22;
  const uint64_t zero = (a.n_rows + groups - 1) / groups;
  const uint64_t zero_blocks = zero < 4096 ? zero : 4096;
  m.sum_blocks = (uint32_t)sum_blocks;
  e = with_dtype(a.in_dtype, [&](auto di) {
    return with_dtype(a.out_dtype, [&](auto dO) {
      grad_sum_kernel<di.value, dO.value><<<(uint32_t)(sum_blocks + zero_blocks), kBlock, 0, s>>>(m);
      return hipGetLastError();
    });
  });
  if (e != hipSuccess || m.nchunks < 2) return e;
  return with_dtype(a.out_dtype, [&](auto dO) {
    grad_join_kernel<dO.value><<<m.sum_blocks, kBlock, 0, s>>>(m);
    return hipGetLastError();
  });
}

}  // namespace ibp
