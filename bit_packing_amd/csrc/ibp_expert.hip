// ibp_expert.hip -- order of tokens by expert: positions sorted by expert number, equal ones
// in their order, and where each expert's begin.
//
// A counting sort.  The experts fit one digit (at most 1024, and one more bin for ids out of
// range), so the ids are read twice and the order written once; no key is ever moved.  Ranks
// come from ballots, not from atomics, so equal ids keep their order.
#include "ibp_device.h"
#include "ibp_ops.h"

namespace ibp {
namespace {

using namespace dev;

constexpr uint32_t kThreads = 1024, kWaves = kThreads / kWave;
constexpr uint32_t kBins = IBP_MAX_EXPERTS + 1;
// Ids that one workgroup sorts, in one launch; ids a workgroup beyond that; workgroups at most.
constexpr uint32_t kOne = 4096, kLeast = 2048, kGroups = 256;

struct Plan {
  uint32_t groups;
  uint32_t per_wave;  // ids a wavefront, a multiple of kWave
};

Plan plan_of(uint64_t n) {
  uint64_t groups = n <= kOne ? 1 : (n + kLeast - 1) / kLeast;
  if (groups > kGroups) groups = kGroups;
  const uint64_t waves = groups * kWaves;
  Plan p{(uint32_t)groups, (uint32_t)(((n + waves - 1) / waves + kWave - 1) / kWave * kWave)};
  return p;
}

__device__ __forceinline__ uint32_t bin_of(const ExpertOrderArgs &a, int64_t id) {
  return id < 0 || (uint64_t)id >= a.experts ? a.experts : (uint32_t)id;
}

// Bins of a workgroup's counts, an even number.
__host__ __device__ constexpr uint32_t row_of(uint32_t experts) { return (experts + 2) / 2 * 2; }

// How many of a workgroup's ids have each bin.
__global__ __launch_bounds__(kThreads) void count_kernel(ExpertOrderArgs a, uint32_t per_wave) {
  __shared__ uint32_t hist[kBins + 1];
  const uint32_t bins = row_of(a.experts);
  for (uint32_t b = threadIdx.x; b < bins; b += kThreads) hist[b] = 0;
  __syncthreads();
  const uint64_t first = (uint64_t)blockIdx.x * per_wave * kWaves, next = first + (uint64_t)per_wave * kWaves;
  const uint64_t end = next < a.n ? next : a.n;
  for (uint64_t j = first + threadIdx.x; j < end; j += kThreads) atomicAdd(&hist[bin_of(a, a.ids[j])], 1u);
  __syncthreads();
  for (uint32_t b = threadIdx.x; b < bins; b += kThreads) a.counts[(uint64_t)blockIdx.x * bins + b] = hist[b];
}

// Each id's place: the ids of smaller bins, those of its bin in earlier workgroups, earlier
// wavefronts, and earlier in the wavefront.  With one workgroup nothing is counted before.
// A thread owns two bins, and as many threads as there are share the workgroups' counts of two
// bins (`pairs`, a power of two, is the threads of one share).
template <bool ONE>
__global__ __launch_bounds__(kThreads) void place_kernel(ExpertOrderArgs a, uint32_t per_wave, uint32_t bits, uint32_t pairs) {
  __shared__ __align__(16) uint32_t off[kWaves][kBins + 3];  // rows end off a multiple of 64 banks
  __shared__ uint4 sums[ONE ? 1 : kThreads];
  __shared__ uint32_t wave_total[kWaves];
  const uint32_t t = threadIdx.x, wave = uniform(t / kWave), lane = lane_id(), bins = row_of(a.experts);
  const uint64_t w0 = ((uint64_t)blockIdx.x * kWaves + wave) * per_wave, w1 = w0 + per_wave;
  const uint64_t end = w1 < a.n ? w1 : a.n;
  // the first ids stay in registers, where their loads are in flight together
  constexpr uint32_t kKept = 4;
  uint32_t kept[kKept];
#pragma unroll
  for (uint32_t k = 0; k < kKept; ++k) {
    const uint64_t j = w0 + k * kWave + lane;
    kept[k] = j < end ? bin_of(a, a.ids[j]) : ~0u;
  }
  uint4 sum = make_uint4(0u, 0u, 0u, 0u);  // of two bins in all workgroups, and in earlier ones
  if constexpr (!ONE) {
    const uint32_t pair = t & (pairs - 1), share = t / pairs, shares = kThreads / pairs;
    const bool in = 2 * pair < bins;
    const uint32_t *counts = a.counts + (in ? 2 * pair : 0);
    constexpr uint32_t kFlight = 16;  // loads in flight: the counts come from L2
    for (uint32_t g0 = share; g0 < gridDim.x; g0 += kFlight * shares) {
      uint2 c[kFlight];
#pragma unroll
      for (uint32_t k = 0; k < kFlight; ++k) {
        const uint32_t g = g0 + k * shares;
        c[k] = g < gridDim.x && in ? *reinterpret_cast<const uint2 *>(counts + (uint64_t)g * bins) : make_uint2(0u, 0u);
      }
#pragma unroll
      for (uint32_t k = 0; k < kFlight; ++k) {
        const bool early = g0 + k * shares < blockIdx.x;
        sum.x += c[k].x;
        sum.y += c[k].y;
        sum.z += early ? c[k].x : 0u;
        sum.w += early ? c[k].y : 0u;
      }
    }
    sums[t] = sum;
  }
  for (uint32_t w = 0; w < kWaves; ++w)
    for (uint32_t b = t; b < bins; b += kThreads) off[w][b] = 0;
  __syncthreads();
#pragma unroll
  for (uint32_t k = 0; k < kKept; ++k)
    if (kept[k] != ~0u) atomicAdd(&off[wave][kept[k]], 1u);
  for (uint64_t j = w0 + kKept * kWave + lane; j < end; j += kWave) atomicAdd(&off[wave][bin_of(a, a.ids[j])], 1u);
  __syncthreads();
  // thread t owns bins 2 t and 2 t + 1
  const bool own = t < pairs && 2 * t < bins;
  uint2 c[kWaves];
#pragma unroll
  for (uint32_t w = 0; w < kWaves; ++w) c[w] = own ? *reinterpret_cast<const uint2 *>(&off[w][2 * t]) : make_uint2(0u, 0u);
  if constexpr (ONE) {
#pragma unroll
    for (uint32_t w = 0; w < kWaves; ++w) {
      sum.x += c[w].x;
      sum.y += c[w].y;
    }
  } else {
    sum = make_uint4(0u, 0u, 0u, 0u);
    if (own) {
      for (uint32_t k = t; k < kThreads; k += pairs) {
        const uint4 v = sums[k];
        sum.x += v.x;
        sum.y += v.y;
        sum.z += v.z;
        sum.w += v.w;
      }
    }
  }
  const uint32_t incl = wave_incl_scan(sum.x + sum.y);
  if (lane == kWave - 1) wave_total[wave] = incl;
  __syncthreads();
  if (own) {
    uint2 at;
    at.x = incl - sum.x - sum.y;
    for (uint32_t w = 0; w < wave; ++w) at.x += wave_total[w];
    at.y = at.x + sum.x;
    if (blockIdx.x == 0) {
      if (2 * t <= a.experts) a.offsets[2 * t] = at.x;
      if (2 * t + 1 <= a.experts) a.offsets[2 * t + 1] = at.y;
      const uint32_t bad = 2 * t == a.experts ? sum.x : (2 * t + 1 == a.experts ? sum.y : 0u);
      if (bad && a.err) atomicOr(a.err, (uint32_t)IBP_DEVERR_BAD_ID);
    }
    at.x += sum.z;
    at.y += sum.w;
#pragma unroll
    for (uint32_t w = 0; w < kWaves; ++w) {
      *reinterpret_cast<uint2 *>(&off[w][2 * t]) = at;
      at.x += c[w].x;
      at.y += c[w].y;
    }
  }
  __syncthreads();
  auto place = [&](uint32_t b, uint64_t j) {
    const bool live = j < end;
    if (!live) b = 0;
    const uint64_t same = same_digit(b, bits, ballot(live));
    const uint32_t rank = count_below(same);
    uint32_t to = 0;
    if (live) to = off[wave][b] + rank;
    wave_lds_sync();
    if (live && rank == 0) off[wave][b] += popc(same);
    wave_lds_sync();
    if (live && to < a.n) a.order[to] = (int64_t)j;  // always, unless the ids change while the call runs
  };
#pragma unroll
  for (uint32_t k = 0; k < kKept; ++k)
    if (w0 + k * kWave < end) place(kept[k], w0 + k * kWave + lane);
  for (uint64_t j0 = w0 + kKept * kWave; j0 < end; j0 += kWave) {
    const uint64_t j = j0 + lane;
    place(j < end ? bin_of(a, a.ids[j]) : 0u, j);
  }
}

}  // namespace

uint64_t expert_order_workspace(uint64_t n, uint32_t experts) {
  const Plan p = plan_of(n);
  return p.groups > 1 ? ((uint64_t)p.groups * row_of(experts) * 4 + 15) / 16 * 16 : 0;
}

hipError_t launch_expert_order(const ExpertOrderArgs &a, hipStream_t s) {
  const Plan p = plan_of(a.n);
  uint32_t bits = 1;
  while (a.experts >> bits) ++bits;
  uint32_t pairs = kWave;
  while (2 * pairs < row_of(a.experts)) pairs *= 2;
  if (p.groups == 1) {
    place_kernel<true><<<1, kThreads, 0, s>>>(a, p.per_wave, bits, pairs);
    return hipGetLastError();
  }
  count_kernel<<<p.groups, kThreads, 0, s>>>(a, p.per_wave);
  const hipError_t e = hipGetLastError();
  if (e != hipSuccess) return e;
  place_kernel<false><<<p.groups, kThreads, 0, s>>>(a, p.per_wave, bits, pairs);
  return hipGetLastError();
}

}  // namespace ibp
