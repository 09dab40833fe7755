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
constexpr uint32_t kOne = 8192;    // ids that one workgroup sorts, in one launch
constexpr uint32_t kLeast = 2048;  // ids a workgroup beyond that
constexpr uint32_t kGroups = 256;  // workgroups at most

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

// How many of a workgroup's ids have each bin.
__global__ __launch_bounds__(kThreads) void count_kernel(ExpertOrderArgs a, uint32_t per_wave) {
  __shared__ uint32_t hist[kBins];
  const uint32_t bins = a.experts + 1;
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
template <bool ONE> __global__ __launch_bounds__(kThreads) void place_kernel(ExpertOrderArgs a, uint32_t per_wave, uint32_t bits) {
  __shared__ uint32_t off[kWaves][kBins + 3];  // rows end off a multiple of 64 banks
  __shared__ uint32_t wave_total[kWaves];
  const uint32_t t = threadIdx.x, wave = uniform(t / kWave), lane = lane_id(), bins = a.experts + 1;
  const uint64_t w0 = ((uint64_t)blockIdx.x * kWaves + wave) * per_wave, w1 = w0 + per_wave;
  const uint64_t end = w1 < a.n ? w1 : a.n;
  for (uint32_t w = 0; w < kWaves; ++w)
    for (uint32_t b = t; b < bins; b += kThreads) off[w][b] = 0;
  __syncthreads();
  for (uint64_t j = w0 + lane; j < end; j += kWave) atomicAdd(&off[wave][bin_of(a, a.ids[j])], 1u);
  __syncthreads();
  // thread b owns bin b, in rounds for more bins than threads
  uint32_t base = 0;  // ids of the bins of the rounds before
  for (uint32_t b0 = 0; b0 < bins; b0 += kThreads) {
    const uint32_t b = b0 + t;
    uint32_t all = 0, early = 0;
    if (b < bins) {
      if constexpr (ONE) {
        for (uint32_t w = 0; w < kWaves; ++w) all += off[w][b];
      } else {
        for (uint32_t g = 0; g < gridDim.x; ++g) {
          const uint32_t c = a.counts[(uint64_t)g * bins + b];
          all += c;
          early += g < blockIdx.x ? c : 0u;
        }
      }
    }
    const uint32_t incl = wave_incl_scan(all);
    if (lane == kWave - 1) wave_total[wave] = incl;
    __syncthreads();
    uint32_t at = base + incl - all;
    for (uint32_t w = 0; w < wave; ++w) at += wave_total[w];
    for (uint32_t w = 0; w < kWaves; ++w) base += wave_total[w];
    if (b < bins) {
      if (blockIdx.x == 0) a.offsets[b] = at;
      if (blockIdx.x == 0 && b == a.experts && all && a.err) atomicOr(a.err, (uint32_t)IBP_DEVERR_BAD_ID);
      at += early;
      for (uint32_t w = 0; w < kWaves; ++w) {
        const uint32_t c = off[w][b];
        off[w][b] = at;
        at += c;
      }
    }
    __syncthreads();
  }
  for (uint64_t j0 = w0; j0 < end; j0 += kWave) {
    const uint64_t j = j0 + lane;
    const bool live = j < end;
    const uint32_t b = live ? bin_of(a, a.ids[j]) : 0u;
    const uint64_t same = same_digit(b, bits, ballot(live));
    const uint32_t rank = count_below(same);
    uint32_t to = 0;
    if (live) to = off[wave][b] + rank;
    wave_lds_sync();
    if (live && rank == 0) off[wave][b] += popc(same);
    wave_lds_sync();
    if (live && to < a.n) a.order[to] = (int64_t)j;  // always, unless the ids change while the call runs
  }
}

}  // namespace

uint64_t expert_order_workspace(uint64_t n, uint32_t experts) {
  const Plan p = plan_of(n);
  return p.groups > 1 ? ((uint64_t)p.groups * (experts + 1) * 4 + 15) / 16 * 16 : 0;
}

hipError_t launch_expert_order(const ExpertOrderArgs &a, hipStream_t s) {
  const Plan p = plan_of(a.n);
  uint32_t bits = 1;
  while (a.experts >> bits) ++bits;
  if (p.groups == 1) {
    place_kernel<true><<<1, kThreads, 0, s>>>(a, p.per_wave, bits);
    return hipGetLastError();
  }
  count_kernel<<<p.groups, kThreads, 0, s>>>(a, p.per_wave);
  const hipError_t e = hipGetLastError();
  if (e != hipSuccess) return e;
  place_kernel<false><<<p.groups, kThreads, 0, s>>>(a, p.per_wave, bits);
  return hipGetLastError();
}

}  // namespace ibp
