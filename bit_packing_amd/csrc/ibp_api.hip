// ibp_api.hip -- the extern "C" entry points declared in include/ibp.h.
//
// Every argument is checked here, on the host, before any HIP call; then the
// launch geometry and the workspace layout are derived and the kernels in
// the other files of this folder are enqueued on the caller's stream.
#include <math.h>
#include <string.h>

#include <atomic>
#include <initializer_list>
#include <mutex>

#include "ibp.h"
#include "ibp_internal.h"
#include "ibp_ops.h"

namespace {

using namespace ibp;

uint64_t full_bits(uint32_t W) { return W >= 64 ? ~0ull : ((1ull << W) - 1ull); }

bool width_ok(uint32_t W) { return W == 16 || W == 32 || W == 64; }

uint32_t log2_if_pow2(uint32_t S) {
  if (S == 0 || (S & (S - 1u))) return kNotPow2;
  uint32_t l = 0;
  while ((1u << l) != S) ++l;
  return l;
}

bool aligned(const void *p, uint64_t a) { return ((uintptr_t)p % a) == 0; }

// x * y, false when the product does not fit 64 bits
bool mul_ok(uint64_t x, uint64_t y, uint64_t *out) { return !__builtin_mul_overflow(x, y, out); }

// Look-back polls of one unpublished predecessor before a compressing tile gives
// up (see lookback_finish); lowered only by tests of that path.
constexpr uint32_t kDefaultWaitLimit = 1u << 20;
std::atomic<uint32_t> g_wait_limit{kDefaultWaitLimit};
constexpr uint64_t kDefaultHalvesMin = 1ull << 23;  // chunks; see ibp_set_halves_min_chunks
std::atomic<uint64_t> g_halves_min{kDefaultHalvesMin};

// Mask/Bitval -> kernel parameters: popcount and the runs of free positions.
bool make_params(const ibp_meta_t *m, CodecParams *p) {
  if (!m || !width_ok(m->W) || m->reserved != 0) return false;
  const uint64_t full = full_bits(m->W);
  if ((m->mask & ~full) || (m->bitval & ~m->mask)) return false;
  memset(p, 0, sizeof(*p));
  p->mask = m->mask;
  p->bitval = m->bitval;
  p->W = m->W;
  p->pc = (uint32_t)__builtin_popcountll(m->mask);
  const uint64_t F = ~m->mask & full;
  uint32_t n = 0, cum = 0;
  for (uint32_t b = 0; b < m->W;) {
    if (!((F >> b) & 1ull)) {
      ++b;
      continue;
    }
    const uint32_t start = b;
    while (b < m->W && ((F >> b) & 1ull)) ++b;
    const uint32_t len = b - start;
    p->runs.pmask[n] = full_bits(len) << cum;
    p->runs.shift[n] = start - cum;
    cum += len;
    ++n;
  }
  p->runs.n = n;
  return true;
}

// Bits per segment can never exceed S * (W + 1); total bits must fit the 62-bit
// look-back value field.
bool total_fits(uint64_t n_chunks, uint32_t W) {
  return n_chunks < (1ull << 55) && n_chunks * (uint64_t)(W + 1) < (1ull << 62);
}

uint32_t meta_blocks(uint64_t n) {
  // about four samples per thread: one round of four in-flight steps per wavefront
  const uint64_t want = (n + (uint64_t)kMetaThreads * 4 - 1) / ((uint64_t)kMetaThreads * 4);
  return (uint32_t)(want < 1 ? 1 : (want > kMetaMaxBlocks ? kMetaMaxBlocks : want));
}

uint32_t enc_segs_per_tile(uint32_t S, bool pos, bool pair, uint32_t W, uint32_t halves = 1, bool big = false) {
  const uint32_t tile = enc_tile_chunks(pos, pair, W, halves, big);
  return S >= tile ? 1u : tile / S;
}

uint64_t enc_tiles(uint64_t n_chunks, uint32_t S, bool pos, bool pair, uint32_t W) {
  const uint64_t nseg = (n_chunks + S - 1) / S;
  const uint32_t G = enc_segs_per_tile(S, pos, pair, W);
  return (nseg + G - 1) / G;
}

uint32_t dec_units_per_tile(uint32_t S) {
  uint32_t G = S >= kDecTileChunks ? 1u : kDecTileChunks / S;
  return G > kDecMaxUnits ? kDecMaxUnits : G;
}

int status_of(hipError_t e) { return e == hipSuccess ? IBP_OK : IBP_ERR_DEVICE; }

// Device-visible address of the byte range [p, p + bytes), or nullptr when the
// range does not lie inside one device allocation or one pinned host allocation.
// Pageable host memory and stray pointers are refused here instead of being
// handed to a kernel, where they would fault the GPU.  Pinned host memory is
// returned through its device mapping (the zero-copy path).
struct Range { const void *p; uint64_t bytes; };

const void *device_range(const void *p, uint64_t bytes, bool *is_host = nullptr, Range *allocation = nullptr) {
  if (is_host) *is_host = false;
  if (bytes == 0) return p;
  if (!p) return nullptr;
  hipPointerAttribute_t at;
  if (hipPointerGetAttributes(&at, p) != hipSuccess) {
    (void)hipGetLastError();
    return nullptr;
  }
  const char *dev;
  if (at.type == hipMemoryTypeDevice || at.type == hipMemoryTypeManaged) {
    dev = static_cast<const char *>(p);
  } else if (at.type == hipMemoryTypeHost && at.devicePointer) {
    if (is_host) *is_host = true;
    const char *hp = at.hostPointer ? static_cast<const char *>(at.hostPointer) : static_cast<const char *>(p);
    dev = static_cast<const char *>(at.devicePointer) + (static_cast<const char *>(p) - hp);
  } else {
    return nullptr;
  }
  // the allocation that holds q must also hold [q, q + bytes): 1 yes, 0 no, -1 unknown
  auto inside = [&](const void *q) -> int {
    hipDeviceptr_t base = nullptr;
    size_t size = 0;
    if (hipMemGetAddressRange(&base, &size, (hipDeviceptr_t)q) != hipSuccess) {
      (void)hipGetLastError();
      return -1;
    }
    const uintptr_t b = (uintptr_t)base, a = (uintptr_t)q;
    if (allocation && at.type == hipMemoryTypeDevice) *allocation = {(const void *)base, size};
    return (a >= b && bytes <= size && a - b <= size - bytes) ? 1 : 0;
  };
  int in = inside(dev);
  // pinned host memory: the range may be known under its host address instead
  if (in < 0 && at.type == hipMemoryTypeHost) in = inside(p);
  return in == 1 ? dev : nullptr;
}

template <typename P> bool view(P *&p, uint64_t bytes, bool *is_host = nullptr) {
  const void *d = device_range(p, bytes, is_host);
  if (bytes && !d) return false;
  p = const_cast<P *>(static_cast<const P *>(d));
  return true;
}

// The views of one call: its tensors often lie in one allocation, which is looked up once
// (a call that packs one row to 8-bit integers: 4.0 us with three look-ups, 3.7 with one).
struct Views {
  Range last = {nullptr, 0};
  template <typename P> bool operator()(P *&p, uint64_t bytes) {
    const uintptr_t at = (uintptr_t)p - (uintptr_t)last.p;
    if (bytes == 0 || (p && bytes <= last.bytes && at <= last.bytes - bytes)) return true;
    const void *d = device_range(p, bytes, nullptr, &last);
    if (!d) return false;
    p = const_cast<P *>(static_cast<const P *>(d));
    return true;
  }
};

// Workspace of ibp_compress_noalloc, for callers that cannot allocate: a file-scope
// device array (each GPU the library runs on holds its own copy until the process
// ends), shared by every such call on that GPU.  Its device address on each GPU is
// resolved once, with that GPU current, by hipGetSymbolAddress; host code uses only
// that address (the array's name is not a device address in host code).
constexpr uint64_t kScratchBytes = IBP_NOALLOC_SCRATCH_BYTES;
constexpr int kMaxDevices = 64;
static __device__ __align__(256) uint8_t scratch[kScratchBytes];
std::mutex g_scratch_mu;
void *g_scratch_ptr[kMaxDevices] = {};

void *scratch_of_current_device() {
  int dev = -1;
  if (hipGetDevice(&dev) != hipSuccess || dev < 0 || dev >= kMaxDevices) {
    (void)hipGetLastError();
    return nullptr;
  }
  std::lock_guard<std::mutex> lock(g_scratch_mu);
  if (!g_scratch_ptr[dev]) {
    void *ptr = nullptr;
    if (hipGetSymbolAddress(&ptr, HIP_SYMBOL(scratch)) != hipSuccess || !ptr) {
      (void)hipGetLastError();
      return nullptr;
    }
    g_scratch_ptr[dev] = ptr;
  }
  return g_scratch_ptr[dev];
}

}  // namespace

extern "C" {

IBP_API const char *ibp_status_str(int status) {
  switch (status) {
    case IBP_OK: return "IBP_OK";
    case IBP_ERR_INVALID_ARG: return "IBP_ERR_INVALID_ARG";
    case IBP_ERR_SIZE: return "IBP_ERR_SIZE";
    case IBP_ERR_CAPACITY: return "IBP_ERR_CAPACITY";
    case IBP_ERR_DEVICE: return "IBP_ERR_DEVICE";
    default: return "IBP_ERR_UNKNOWN";
  }
}

IBP_API uint32_t ibp_set_wait_limit(uint32_t polls) {
  return g_wait_limit.exchange(polls == 0xFFFFFFFFu ? kDefaultWaitLimit : polls);
}

IBP_API uint64_t ibp_set_halves_min_chunks(uint64_t n_chunks) {
  return g_halves_min.exchange(n_chunks == ~0ull ? kDefaultHalvesMin : n_chunks);
}

IBP_API uint64_t ibp_num_segments(uint64_t n_chunks, uint32_t S) {
  return S ? (n_chunks + S - 1) / S : 0;
}

IBP_API uint64_t ibp_max_stream_bytes(uint64_t n_chunks, uint32_t W) {
  const uint64_t bytes = (n_chunks * (uint64_t)(W + 1) + 7) / 8;
  return (bytes + 15) & ~15ull;
}

IBP_API uint64_t ibp_stream_bytes(uint64_t total_bits) { return (((total_bits + 7) / 8) + 15) & ~15ull; }

IBP_API uint64_t ibp_metadata_workspace_bytes(uint64_t n_sample_chunks, uint32_t W) {
  const uint64_t w = width_ok(W) ? W : 64;
  return ((uint64_t)meta_blocks(n_sample_chunks) * w + 66) * 8;
}

IBP_API uint64_t ibp_compress_workspace_bytes(uint64_t n_chunks, uint32_t S) {
  if (S == 0) return 0;
  const uint64_t t = enc_tiles(n_chunks, S, true, false, 32);  // the smallest tiles (position metadata, W > 16)
  return t ? 8 + 8 * (status_words(t) + t) : 8;  // control, status words, hand-over words
}

IBP_API int ibp_build_metadata(const void *d_samples, uint64_t n_sample_chunks, uint32_t W, double T,
                               ibp_meta_t *meta_out, uint64_t *counts_out, void *d_workspace,
                               uint64_t workspace_bytes, void *hip_stream) {
  if (!width_ok(W) || !meta_out || !d_workspace || !(T > 0.5 && T <= 1.0)) return IBP_ERR_INVALID_ARG;
  if (n_sample_chunks == 0 || !d_samples || !aligned(d_samples, W / 8) || !aligned(d_workspace, 8))
    return IBP_ERR_INVALID_ARG;
  if (n_sample_chunks >= (1ull << 40)) return IBP_ERR_SIZE;
  if (workspace_bytes < ibp_metadata_workspace_bytes(n_sample_chunks, W)) return IBP_ERR_CAPACITY;
  if (!view(d_samples, n_sample_chunks * (W / 8)) || !view(d_workspace, ibp_metadata_workspace_bytes(n_sample_chunks, W)))
    return IBP_ERR_INVALID_ARG;
  hipStream_t s = static_cast<hipStream_t>(hip_stream);
  MetaArgs a;
  a.in = d_samples;
  a.n = n_sample_chunks;
  a.W = W;
  a.blocks = meta_blocks(n_sample_chunks);
  a.partial = static_cast<uint64_t *>(d_workspace);
  a.result = a.partial + (uint64_t)a.blocks * W;
  // k = ceil(round(T * 10^6) * n / 10^6), exactly, in 128-bit integers
  const uint64_t tppm = (uint64_t)(T * 1e6 + 0.5);
  const unsigned __int128 num = (unsigned __int128)tppm * n_sample_chunks;
  a.k = (uint64_t)((num + 999999u) / 1000000u);
  hipError_t e = launch_meta(a, s);
  if (e != hipSuccess) return IBP_ERR_DEVICE;
  uint64_t host[66];
  e = hipMemcpyAsync(host, a.result, sizeof(host), hipMemcpyDeviceToHost, s);
  if (e != hipSuccess) return IBP_ERR_DEVICE;
  e = hipStreamSynchronize(s);
  if (e != hipSuccess) return IBP_ERR_DEVICE;
  meta_out->W = W;
  meta_out->reserved = 0;
  meta_out->mask = host[64];
  meta_out->bitval = host[65];
  if (counts_out)
    for (uint32_t b = 0; b < W; ++b) counts_out[b] = host[b];
  return IBP_OK;
}

// ws_is_scratch: d_workspace is this library's own device array (ibp_compress_noalloc),
// known to be device memory of kScratchBytes bytes; it is not looked up.
static int compress_common(const CodecParams &p, const uint64_t *pmask, const uint64_t *pbitval, const void *d_in,
                           uint64_t n_bytes, uint32_t S, void *d_stream, uint64_t stream_capacity,
                           uint64_t *d_offsets, void *d_workspace, uint64_t workspace_bytes, uint32_t *d_err_word,
                           void *hip_stream, bool ws_is_scratch = false) {
  if (S == 0 || S > IBP_MAX_S || !d_offsets) return IBP_ERR_INVALID_ARG;
  const uint32_t cb = p.W / 8;
  if (n_bytes % cb) return IBP_ERR_SIZE;
  const uint64_t n = n_bytes / cb;
  if (n && (!d_in || !d_stream || !d_workspace)) return IBP_ERR_INVALID_ARG;
  if (!aligned(d_in, cb) || !aligned(d_stream, 16) || !aligned(d_offsets, 8) || !aligned(d_workspace, 8))
    return IBP_ERR_INVALID_ARG;
  if (!total_fits(n, p.W)) return IBP_ERR_SIZE;
  if (stream_capacity < ibp_max_stream_bytes(n, p.W)) return IBP_ERR_CAPACITY;
  if (workspace_bytes < ibp_compress_workspace_bytes(n, S)) return IBP_ERR_CAPACITY;
  const uint64_t nseg = (n + S - 1) / S;
  if (!view(d_in, n_bytes) || !view(d_stream, ibp_max_stream_bytes(n, p.W)) || !view(d_offsets, 8 * (nseg + 1)) ||
      (!ws_is_scratch && !view(d_workspace, n ? ibp_compress_workspace_bytes(n, S) : 0)) ||
      !view(d_err_word, d_err_word ? 4 : 0))
    return IBP_ERR_INVALID_ARG;
  hipStream_t s = static_cast<hipStream_t>(hip_stream);
  if (n == 0) return status_of(launch_zero(d_offsets, 1, s));  // offset table = {0}
  EncodeArgs a;
  a.pmask = pmask;
  a.pbitval = pbitval;
  a.in = d_in;
  a.stream = static_cast<uint32_t *>(d_stream);
  a.off = d_offsets;
  a.control = static_cast<uint32_t *>(d_workspace);
  a.status = reinterpret_cast<uint64_t *>(static_cast<uint8_t *>(d_workspace) + 8);
  // W = 16 with one Mask reads chunk pairs as 32-bit words when the segments are
  // whole 64-chunk blocks and the input allows it
  a.pair = (p.W == 16 && !pmask && S % kWave == 0 && aligned(d_in, 4)) ? 1u : 0u;
  a.halves = n >= g_halves_min.load() ? enc_halves(pmask != nullptr, a.pair != 0u, p.W, S) : 1u;
  a.big = !pmask && enc_big(p.W, a.halves, p.pc) ? 1u : 0u;
  a.G = enc_segs_per_tile(S, pmask != nullptr, a.pair != 0u, p.W, a.halves, a.big != 0u);
  a.ntiles = (nseg + a.G - 1) / a.G;  // at most the workspace's tile count (its tiles are the smallest)
  a.st_lg = status_lg(a.ntiles);
  a.tails = a.status + status_words(a.ntiles);
  a.err = d_err_word;
  a.n_chunks = n;
  a.nseg = nseg;
  a.S = S;
  a.s_log2 = log2_if_pow2(S);
  a.tile_chunks = a.G * S;
  if (a.halves == 2 && a.tile_chunks != enc_tile_chunks(pmask != nullptr, false, p.W, 2, a.big != 0u))
    return IBP_ERR_INVALID_ARG;
  // image (one half's when halves == 2) from the 16-byte block of the first bit
  a.obuf_dw = ((127 + a.tile_chunks / a.halves * (p.W + 1) + 31) / 32 + 2 + 3) & ~3u;
  a.wait_limit = g_wait_limit.load();
  return status_of(launch_encode(a, p, s));
}

IBP_API int ibp_compress(const ibp_meta_t *meta, const void *d_in, uint64_t n_bytes, uint32_t S,
                         void *d_stream, uint64_t stream_capacity, uint64_t *d_offsets,
                         void *d_workspace, uint64_t workspace_bytes, uint32_t *d_err_word,
                         void *hip_stream) {
  CodecParams p;
  if (!make_params(meta, &p)) return IBP_ERR_INVALID_ARG;
  return compress_common(p, nullptr, nullptr, d_in, n_bytes, S, d_stream, stream_capacity, d_offsets, d_workspace,
                         workspace_bytes, d_err_word, hip_stream);
}

IBP_API int ibp_compress_noalloc(const ibp_meta_t *meta, const void *d_in, uint64_t n_bytes, uint32_t S,
                                 void *d_stream, uint64_t stream_capacity, uint64_t *d_offsets,
                                 uint32_t *d_err_word, void *hip_stream) {
  CodecParams p;
  if (!make_params(meta, &p)) return IBP_ERR_INVALID_ARG;
  if (S == 0 || S > IBP_MAX_S) return IBP_ERR_INVALID_ARG;
  const uint32_t cb = p.W / 8;
  if (n_bytes % cb) return IBP_ERR_SIZE;
  if (!total_fits(n_bytes / cb, p.W)) return IBP_ERR_SIZE;
  if (ibp_compress_workspace_bytes(n_bytes / cb, S) > kScratchBytes) return IBP_ERR_CAPACITY;
  void *ws = nullptr;
  if (n_bytes) {
    ws = scratch_of_current_device();
    if (!ws) return IBP_ERR_DEVICE;
  }
  return compress_common(p, nullptr, nullptr, d_in, n_bytes, S, d_stream, stream_capacity, d_offsets, ws,
                         kScratchBytes, d_err_word, hip_stream, true);
}

// Position-dependent metadata: W/S checks, device tables of S words each.
static bool pos_params(const ibp_pos_meta_t *m, CodecParams *p, const uint64_t **mask, const uint64_t **bitval) {
  if (!m || !width_ok(m->W) || m->S == 0 || m->S > IBP_MAX_S || !m->mask || !m->bitval) return false;
  if (!aligned(m->mask, 8) || !aligned(m->bitval, 8)) return false;
  *mask = m->mask;
  *bitval = m->bitval;
  if (!view(*mask, 8ull * m->S) || !view(*bitval, 8ull * m->S)) return false;
  memset(p, 0, sizeof(*p));
  p->W = m->W;
  return true;
}

IBP_API uint64_t ibp_metadata_pos_workspace_bytes(uint32_t S, uint32_t W) {
  const uint64_t w = width_ok(W) ? W : 64;
  return 8ull * S * w;
}

IBP_API int ibp_build_metadata_pos(const void *d_samples, uint64_t n_rows, uint32_t S, uint32_t W, double T,
                                   uint64_t *d_mask, uint64_t *d_bitval, uint64_t *counts_out, void *d_workspace,
                                   uint64_t workspace_bytes, void *hip_stream) {
  if (!width_ok(W) || S == 0 || S > IBP_MAX_S || !(T > 0.5 && T <= 1.0)) return IBP_ERR_INVALID_ARG;
  if (n_rows == 0 || !d_samples || !d_mask || !d_bitval || !d_workspace) return IBP_ERR_INVALID_ARG;
  if (!aligned(d_samples, W / 8) || !aligned(d_mask, 8) || !aligned(d_bitval, 8) || !aligned(d_workspace, 8))
    return IBP_ERR_INVALID_ARG;
  if (n_rows >= (1ull << 32) || n_rows * S >= (1ull << 40)) return IBP_ERR_SIZE;
  if (workspace_bytes < ibp_metadata_pos_workspace_bytes(S, W)) return IBP_ERR_CAPACITY;
  if (!view(d_samples, n_rows * S * (W / 8)) || !view(d_mask, 8ull * S) || !view(d_bitval, 8ull * S) ||
      !view(d_workspace, ibp_metadata_pos_workspace_bytes(S, W)))
    return IBP_ERR_INVALID_ARG;
  hipStream_t s = static_cast<hipStream_t>(hip_stream);
  MetaArgs a;
  a.in = d_samples;
  a.n = n_rows;
  a.W = W;
  a.blocks = 0;
  a.partial = static_cast<uint64_t *>(d_workspace);
  a.result = nullptr;
  const uint64_t tppm = (uint64_t)(T * 1e6 + 0.5);
  const unsigned __int128 num = (unsigned __int128)tppm * n_rows;
  a.k = (uint64_t)((num + 999999u) / 1000000u);
  hipError_t e = launch_meta_pos(a, S, d_mask, d_bitval, s);
  if (e != hipSuccess) return IBP_ERR_DEVICE;
  if (counts_out) {
    e = hipMemcpyAsync(counts_out, a.partial, 8ull * S * W, hipMemcpyDeviceToHost, s);
    if (e == hipSuccess) e = hipStreamSynchronize(s);
    if (e != hipSuccess) return IBP_ERR_DEVICE;
  }
  return IBP_OK;
}

IBP_API int ibp_compress_pos(const ibp_pos_meta_t *meta, const void *d_in, uint64_t n_bytes, void *d_stream,
                             uint64_t stream_capacity, uint64_t *d_offsets, void *d_workspace,
                             uint64_t workspace_bytes, uint32_t *d_err_word, void *hip_stream) {
  CodecParams p;
  const uint64_t *pm, *pb;
  if (!pos_params(meta, &p, &pm, &pb)) return IBP_ERR_INVALID_ARG;
  return compress_common(p, pm, pb, d_in, n_bytes, meta->S, d_stream, stream_capacity, d_offsets,
                         d_workspace, workspace_bytes, d_err_word, hip_stream);
}

static int decode_common(const CodecParams &p, const uint64_t *pmask, const uint64_t *pbitval, const void *stream_in,
                         uint64_t stream_bytes, const uint64_t *d_offsets, uint64_t nseg, uint32_t S,
                         const int64_t *d_ids, uint64_t n_units, uint64_t n_chunks, void *d_out,
                         uint32_t *d_err_word, void *hip_stream, bool gather) {
  if (S == 0 || S > IBP_MAX_S || !d_offsets) return IBP_ERR_INVALID_ARG;
  const uint32_t cb = p.W / 8;
  if (n_chunks && (!d_out || !stream_in)) return IBP_ERR_INVALID_ARG;
  if (gather && n_units && !d_ids) return IBP_ERR_INVALID_ARG;
  if (!aligned(stream_in, 16) || !aligned(d_out, cb) || !aligned(d_offsets, 8) || !aligned(d_ids, 8))
    return IBP_ERR_INVALID_ARG;
  if (nseg >= (1ull << 55) / S) return IBP_ERR_SIZE;  // keeps 8 (nseg + 1) and nseg S exact
  if (!total_fits(n_chunks, p.W) || (gather && !total_fits(nseg * (uint64_t)S, p.W))) return IBP_ERR_SIZE;
  if (n_units == 0) return IBP_OK;
  bool host_stream = false;
  if (!view(stream_in, stream_bytes, &host_stream) || !view(d_offsets, 8 * (nseg + 1)) || !view(d_ids, gather ? 8 * n_units : 0) ||
      !view(d_out, n_chunks * cb) || !view(d_err_word, d_err_word ? 4 : 0))
    return IBP_ERR_INVALID_ARG;
  DecodeArgs a;
  a.pmask = pmask;
  a.pbitval = pbitval;
  a.stream = static_cast<const uint8_t *>(stream_in);
  a.stream_bytes = stream_bytes;
  a.off = d_offsets;
  a.ids = d_ids;
  a.out = d_out;
  a.err = d_err_word;
  a.n_chunks = n_chunks;
  a.n_units = n_units;
  a.nseg = nseg;
  a.S = S;
  a.s_log2 = log2_if_pow2(S);
  // Rows read over PCIe go one per wavefront: more independent read streams keep
  // more host reads in flight.  From HBM a wavefront takes about 512 chunks of a
  // contiguous stream, and about 1024 chunks, at most kGatherMaxRows rows, of a
  // gather (its dependent id -> offset -> row reads favour one wave generation).
  // A contiguous stream with one Mask takes 512 chunks per wavefront; from 2^24
  // chunks on, 512 * 64 / W (the same ~4 KB of staging at every W), which spreads
  // the per-tile setup over more chunks (sparse W = 32 data: 197 -> 159 us per
  // 128M chunks; W = 16: 969 -> 865 us per 1G chunks), while smaller inputs keep
  // more wavefronts.
  if (gather) {
    a.G = host_stream ? 1u : (S >= 2 * kDecTileChunks / kGatherMaxRows ? (S >= 2 * kDecTileChunks ? 1u : 2 * kDecTileChunks / S)
                                                                       : kGatherMaxRows);
  } else if (pmask) {
    a.G = dec_units_per_tile(S);
  } else {
    const uint32_t tile = n_chunks >= (1ull << 24) ? kDecTileChunks * (64u / p.W) : kDecTileChunks;
    a.G = S >= tile ? 1u : (tile / S > kDecMaxUnits ? kDecMaxUnits : tile / S);
  }
  const uint32_t tile_chunks = a.G * S;
  if (gather) {
    a.slot_dw = ((S * (p.W + 1) + 127) / 128 + 1) * 4;
    a.sb_magic = (uint32_t)(((1ull << 32) + a.slot_dw / 4 - 1) / (a.slot_dw / 4));
    a.stage_dw = a.G * a.slot_dw + 4;
  } else {
    a.slot_dw = 0;
    a.sb_magic = 0;
    a.stage_dw = 4 * ((tile_chunks * (p.W + 1) + 254) / 128) + 8;
  }
  uint32_t per_unit = 3 * a.G;
  if (gather) per_unit += (a.G & 1u) + 3 * a.G;  // 8-byte aligned first-block table + block counts
  a.wave_dw = (a.stage_dw + per_unit + 3) & ~3u;
  if (pmask) return status_of(launch_decode_pos(a, p, static_cast<hipStream_t>(hip_stream)));
  return status_of(launch_decode(a, p, gather, static_cast<hipStream_t>(hip_stream)));
}

IBP_API int ibp_decompress(const ibp_meta_t *meta, const void *stream_in, uint64_t stream_bytes,
                           const uint64_t *d_offsets, uint64_t n_chunks, uint32_t S, void *d_out,
                           uint32_t *d_err_word, void *hip_stream) {
  CodecParams p;
  if (!make_params(meta, &p)) return IBP_ERR_INVALID_ARG;
  const uint64_t nseg = ibp_num_segments(n_chunks, S);
  return decode_common(p, nullptr, nullptr, stream_in, stream_bytes, d_offsets, nseg, S, nullptr, nseg, n_chunks,
                       d_out, d_err_word, hip_stream, false);
}

IBP_API int ibp_decompress_pos(const ibp_pos_meta_t *meta, const void *stream_in, uint64_t stream_bytes,
                               const uint64_t *d_offsets, uint64_t n_chunks, void *d_out, uint32_t *d_err_word,
                               void *hip_stream) {
  CodecParams p;
  const uint64_t *pm, *pb;
  if (!pos_params(meta, &p, &pm, &pb)) return IBP_ERR_INVALID_ARG;
  const uint64_t nseg = ibp_num_segments(n_chunks, meta->S);
  return decode_common(p, pm, pb, stream_in, stream_bytes, d_offsets, nseg, meta->S, nullptr, nseg,
                       n_chunks, d_out, d_err_word, hip_stream, false);
}

IBP_API int ibp_decompress_gather(const ibp_meta_t *meta, const void *stream_in, uint64_t stream_bytes,
                                  const uint64_t *d_offsets, uint64_t n_segments, uint32_t S,
                                  const int64_t *d_ids, uint64_t n_ids, void *d_out,
                                  uint32_t *d_err_word, void *hip_stream) {
  CodecParams p;
  if (!make_params(meta, &p)) return IBP_ERR_INVALID_ARG;
  if (S != 0 && n_ids > (1ull << 55) / S) return IBP_ERR_SIZE;
  return decode_common(p, nullptr, nullptr, stream_in, stream_bytes, d_offsets, n_segments, S, d_ids, n_ids,
                       n_ids * (uint64_t)S, d_out, d_err_word, hip_stream, true);
}

IBP_API int ibp_gather_raw(const void *src, uint64_t row_bytes, uint64_t n_rows, const int64_t *d_ids,
                           uint64_t n_ids, void *d_out, uint32_t *d_err_word, void *hip_stream) {
  if (row_bytes == 0 || row_bytes % 16) return IBP_ERR_SIZE;
  uint64_t src_bytes = 0, out_bytes = 0, id_bytes = 0;
  if (!mul_ok(row_bytes, n_rows, &src_bytes) || !mul_ok(row_bytes, n_ids, &out_bytes) || !mul_ok(8, n_ids, &id_bytes))
    return IBP_ERR_SIZE;
  if (n_ids && (!src || !d_ids || !d_out)) return IBP_ERR_INVALID_ARG;
  if (!aligned(src, 16) || !aligned(d_out, 16) || !aligned(d_ids, 8)) return IBP_ERR_INVALID_ARG;
  if (n_ids == 0) return IBP_OK;
  if (n_rows == 0) return IBP_ERR_SIZE;  // every id would be out of range
  if (!view(src, src_bytes) || !view(d_ids, id_bytes) || !view(d_out, out_bytes) ||
      !view(d_err_word, d_err_word ? 4 : 0))
    return IBP_ERR_INVALID_ARG;
  RawGatherArgs a;
  a.src = static_cast<const uint8_t *>(src);
  a.ids = d_ids;
  a.out = static_cast<uint8_t *>(d_out);
  a.err = d_err_word;
  a.row_blocks = row_bytes / 16;
  a.n_rows = n_rows;
  a.n_ids = n_ids;
  return status_of(launch_raw_gather(a, static_cast<hipStream_t>(hip_stream)));
}

}  // extern "C"

// ------------------------------------------------------------------ fixed-slot layout

extern "C" {

IBP_API uint64_t ibp_slot_flag_words(uint64_t n_rows) { return (n_rows + 63) / 64; }

IBP_API int ibp_compress_slots(const ibp_meta_t *meta, const void *d_in, uint64_t n_rows, uint32_t S,
                               void *slots, uint64_t slots_bytes, uint64_t *d_flags, uint32_t *d_err_word,
                               void *hip_stream) {
  CodecParams p;
  if (!make_params(meta, &p) || S == 0 || S > IBP_MAX_S) return IBP_ERR_INVALID_ARG;
  const uint64_t row_bytes = (uint64_t)S * (p.W / 8);
  if (row_bytes % 16) return IBP_ERR_SIZE;
  if (n_rows && (!d_in || !slots || !d_flags)) return IBP_ERR_INVALID_ARG;
  if (!aligned(d_in, 16) || !aligned(slots, 16) || !aligned(d_flags, 8)) return IBP_ERR_INVALID_ARG;
  if (n_rows >= (1ull << 40)) return IBP_ERR_SIZE;
  if (slots_bytes < n_rows * row_bytes) return IBP_ERR_CAPACITY;
  if (n_rows == 0) return IBP_OK;
  bool flags_host = false;
  if (!view(d_in, n_rows * row_bytes) || !view(slots, n_rows * row_bytes) ||
      !view(d_flags, 8 * ibp_slot_flag_words(n_rows), &flags_host) || flags_host ||
      !view(d_err_word, d_err_word ? 4 : 0))
    return IBP_ERR_INVALID_ARG;
  SlotArgs a{};
  a.in = d_in;
  a.slots = static_cast<uint8_t *>(slots);
  a.flags = d_flags;
  a.err = d_err_word;
  a.n_rows = n_rows;
  a.n_units = n_rows;
  a.S = S;
  a.s_log2 = log2_if_pow2(S);
  a.G = dec_units_per_tile(S);
  a.row_bytes = (uint32_t)row_bytes;
  a.img_dw = ((S * (p.W + 1) + 31) / 32 + 2 + 3) & ~3u;
  a.wave_dw = (a.G * a.img_dw + a.G + 1 + 3) & ~3u;
  return status_of(launch_encode_slots(a, p, static_cast<hipStream_t>(hip_stream)));
}

IBP_API int ibp_decompress_gather_slots(const ibp_meta_t *meta, const void *slots, uint64_t slots_bytes,
                                        uint64_t n_rows, uint32_t S, const uint64_t *d_flags, const int64_t *d_ids,
                                        uint64_t n_ids, void *d_out, uint32_t *d_err_word, void *hip_stream) {
  CodecParams p;
  if (!make_params(meta, &p) || S == 0 || S > IBP_MAX_S) return IBP_ERR_INVALID_ARG;
  const uint64_t row_bytes = (uint64_t)S * (p.W / 8);
  if (row_bytes % 16) return IBP_ERR_SIZE;
  if (n_ids && (!slots || !d_flags || !d_ids || !d_out)) return IBP_ERR_INVALID_ARG;
  if (!aligned(slots, 16) || !aligned(d_out, 16) || !aligned(d_flags, 8) || !aligned(d_ids, 8))
    return IBP_ERR_INVALID_ARG;
  if (n_rows >= (1ull << 40) || n_ids >= (1ull << 40)) return IBP_ERR_SIZE;
  if (slots_bytes < n_rows * row_bytes) return IBP_ERR_CAPACITY;
  if (n_ids == 0) return IBP_OK;
  bool slots_host = false, flags_host = false;
  if (!view(slots, n_rows * row_bytes, &slots_host) || !view(d_flags, 8 * ibp_slot_flag_words(n_rows), &flags_host) ||
      flags_host || !view(d_ids, 8 * n_ids) || !view(d_out, n_ids * row_bytes) ||
      !view(d_err_word, d_err_word ? 4 : 0))
    return IBP_ERR_INVALID_ARG;
  SlotArgs a{};
  a.slots = static_cast<uint8_t *>(const_cast<void *>(slots));
  a.flags = const_cast<uint64_t *>(d_flags);
  a.ids = d_ids;
  a.out = d_out;
  a.err = d_err_word;
  a.n_rows = n_rows;
  a.n_units = n_ids;
  a.S = S;
  a.s_log2 = log2_if_pow2(S);
  a.G = slots_host ? 1u : dec_units_per_tile(S);  // one row per wavefront over PCIe, as for the packed gather
  a.row_bytes = (uint32_t)row_bytes;
  const uint32_t row_blocks = (uint32_t)(row_bytes / 16);
  a.img_dw = row_blocks * 4 + 4;
  // First round of loads: the blocks of the shortest compressed row (every chunk
  // matching: S + S (W - popcount(Mask)) bits), at least its header and four
  // blocks, rounded up to whole 128-byte lines of the slot when slots start on
  // lines (host memory is read in 128-byte requests, so the rest of a line costs
  // nothing).  A row longer than that takes a second round.  When most rows are
  // near the shortest length, as on dense data, the slot is read in one round.
  {
    const uint32_t min_bits = S + S * (p.W - p.pc);
    uint32_t h = (min_bits + 127) / 128;
    const uint32_t hdr = (S + 127) / 128;
    if (h < hdr) h = hdr;
    if (h < 4) h = 4;
    if (row_bytes % 128 == 0) h = (h + 7) & ~7u;
    a.head_blocks = h < row_blocks ? h : row_blocks;
  }
  a.wave_dw = (a.G * a.img_dw + 8 * a.G + (a.G & 1u) + 3) & ~3u;
  return status_of(launch_decode_slots(a, p, static_cast<hipStream_t>(hip_stream)));
}

// ------------------------------------------------------------------ comparison codec: BF16 exponent coding

// Mass of BF16 exponent e under N(0, sigma^2): |x| in [2^(e-127), 2^(e-126)) for a
// normal exponent, |x| < 2^-126 for e = 0 (zero and subnormals), none for e = 255.
static double zip_exponent_mass(int e, double sigma) {
  const double d = sigma * sqrt(2.0);
  if (e == 0) return erf(ldexp(1.0, -126) / d);
  if (e == 255) return 0.0;
  return erf(ldexp(1.0, e - 126) / d) - erf(ldexp(1.0, e - 127) / d);
}

IBP_API int ibp_zip_table_from_sigma(double sigma, uint8_t *table_out) {
  if (!table_out || !(sigma > 0.0) || !isfinite(sigma)) return IBP_ERR_INVALID_ARG;
  double mass[256];
  for (int e = 0; e < 256; ++e) mass[e] = zip_exponent_mass(e, sigma);
  bool taken[256] = {false};
  for (int k = 0; k < 7; ++k) {  // largest mass first; equal masses: smaller exponent first
    int best = -1;
    for (int e = 0; e < 256; ++e)
      if (!taken[e] && (best < 0 || mass[e] > mass[best])) best = e;
    taken[best] = true;
    table_out[k] = (uint8_t)best;
  }
  return IBP_OK;
}

IBP_API uint64_t ibp_zip_blocks(uint64_t n) { return (n + kZipBlock - 1) / kZipBlock; }
IBP_API uint64_t ibp_zip_codes_bytes(uint64_t n) { return ibp_zip_blocks(n) * (3 * kZipBlock / 8); }
IBP_API uint64_t ibp_zip_workspace_bytes(uint64_t n) {
  // control word, then the look-back status words of the compressor's workgroups
  return n ? 8 + 8 * status_words((ibp_zip_blocks(n) + kZipWG - 1) / kZipWG) : 8;
}

static bool zip_table_ok(const uint8_t *t) {
  if (!t) return false;
  for (int a = 0; a < 7; ++a)
    for (int b = a + 1; b < 7; ++b)
      if (t[a] == t[b]) return false;
  return true;
}

IBP_API int ibp_zip_compress(const uint8_t *table, const void *d_in, uint64_t n, uint8_t *d_sm, uint8_t *d_codes,
                             uint8_t *d_esc, uint64_t esc_capacity, uint64_t *d_eoff, void *d_workspace,
                             uint64_t workspace_bytes, uint32_t *d_err_word, void *hip_stream) {
  if (!zip_table_ok(table) || !d_eoff) return IBP_ERR_INVALID_ARG;
  if (n >= (1ull << 40)) return IBP_ERR_SIZE;
  if (n && (!d_in || !d_sm || !d_codes || !d_esc || !d_workspace)) return IBP_ERR_INVALID_ARG;
  if (!aligned(d_in, 16) || !aligned(d_sm, 8) || !aligned(d_eoff, 8) || !aligned(d_workspace, 8))
    return IBP_ERR_INVALID_ARG;
  if (esc_capacity < n || workspace_bytes < ibp_zip_workspace_bytes(n)) return IBP_ERR_CAPACITY;
  const uint64_t nblk = ibp_zip_blocks(n);
  if (!view(d_in, 2 * n) || !view(d_sm, n) || !view(d_codes, ibp_zip_codes_bytes(n)) || !view(d_esc, n) ||
      !view(d_eoff, 8 * (nblk + 1)) || !view(d_workspace, n ? ibp_zip_workspace_bytes(n) : 0) ||
      !view(d_err_word, d_err_word ? 4 : 0))
    return IBP_ERR_INVALID_ARG;
  hipStream_t s = static_cast<hipStream_t>(hip_stream);
  if (n == 0) return status_of(launch_zero(d_eoff, 1, s));
  ZipArgs a;
  memset(&a, 0, sizeof(a));
  a.in = static_cast<const uint16_t *>(d_in);
  a.sm = d_sm;
  a.codes = d_codes;
  a.esc = d_esc;
  a.eoff = d_eoff;
  a.control = static_cast<uint32_t *>(d_workspace);
  a.status = reinterpret_cast<uint64_t *>(static_cast<uint8_t *>(d_workspace) + 8);
  a.err = d_err_word;
  a.n = n;
  a.nblk = nblk;
  for (int k = 0; k < 7; ++k) a.table[k] = table[k];
  a.wait_limit = g_wait_limit.load();
  a.st_lg = status_lg((nblk + kZipWG - 1) / kZipWG);
  return status_of(launch_zip_encode(a, s));
}

IBP_API int ibp_zip_decompress(const uint8_t *table, const uint8_t *d_sm, const uint8_t *d_codes,
                               const uint8_t *d_esc, uint64_t esc_bytes, const uint64_t *d_eoff, uint64_t n,
                               void *d_out, uint32_t *d_err_word, void *hip_stream) {
  if (!zip_table_ok(table) || !d_eoff) return IBP_ERR_INVALID_ARG;
  if (n >= (1ull << 40)) return IBP_ERR_SIZE;
  if (n && (!d_sm || !d_codes || !d_out)) return IBP_ERR_INVALID_ARG;
  if (esc_bytes && !d_esc) return IBP_ERR_INVALID_ARG;
  if (!aligned(d_out, 16) || !aligned(d_sm, 8) || !aligned(d_eoff, 8)) return IBP_ERR_INVALID_ARG;
  const uint64_t nblk = ibp_zip_blocks(n);
  if (!view(d_sm, n) || !view(d_codes, ibp_zip_codes_bytes(n)) || !view(d_esc, esc_bytes) ||
      !view(d_eoff, 8 * (nblk + 1)) || !view(d_out, 2 * n) || !view(d_err_word, d_err_word ? 4 : 0))
    return IBP_ERR_INVALID_ARG;
  if (n == 0) return IBP_OK;
  ZipArgs a;
  memset(&a, 0, sizeof(a));
  a.out = static_cast<uint16_t *>(d_out);
  a.sm = const_cast<uint8_t *>(d_sm);
  a.codes = const_cast<uint8_t *>(d_codes);
  a.esc = const_cast<uint8_t *>(d_esc);
  a.esc_bytes = esc_bytes;
  a.eoff = const_cast<uint64_t *>(d_eoff);
  a.err = d_err_word;
  a.n = n;
  a.nblk = nblk;
  for (int k = 0; k < 7; ++k) a.table[k] = table[k];
  return status_of(launch_zip_decode(a, static_cast<hipStream_t>(hip_stream)));
}

// ------------------------------------------------------------------ language-model operators

static uint64_t dtype_size(int dtype) { return dtype == IBP_F32 ? 4 : 2; }
static bool dtype_ok(int dtype) { return dtype == IBP_F32 || dtype == IBP_F16 || dtype == IBP_BF16; }

// Bytes of rows x cols elements; false when they do not fit 64 bits.
static bool matrix_bytes(uint64_t rows, uint64_t cols, uint64_t size, uint64_t *out) {
  return mul_ok(rows, cols, out) && mul_ok(*out, size, out);
}

IBP_API int ibp_embedding_lookup(const void *table, int table_dtype, uint64_t n_rows, uint32_t dim,
                                 const int64_t *d_ids, uint64_t n_ids, float scale, void *d_out, int out_dtype,
                                 uint32_t *d_err_word, void *hip_stream) {
  if (!dtype_ok(table_dtype) || !dtype_ok(out_dtype)) return IBP_ERR_INVALID_ARG;
  if (dim > IBP_MAX_COLS || (n_rows == 0 && n_ids > 0)) return IBP_ERR_SIZE;
  uint64_t tb, ib, ob;
  if (!matrix_bytes(n_rows, dim, dtype_size(table_dtype), &tb) || !mul_ok(n_ids, 8, &ib) ||
      !matrix_bytes(n_ids, dim, dtype_size(out_dtype), &ob))
    return IBP_ERR_SIZE;
  if (n_ids == 0 || dim == 0) return IBP_OK;
  if (!table || !d_ids || !d_out || !aligned(table, dtype_size(table_dtype)) || !aligned(d_ids, 8) ||
      !aligned(d_out, dtype_size(out_dtype)) || !aligned(d_err_word, 4))
    return IBP_ERR_INVALID_ARG;
  Views see;
  if (!see(table, tb) || !see(d_ids, ib) || !see(d_out, ob) || !see(d_err_word, d_err_word ? 4 : 0))
    return IBP_ERR_INVALID_ARG;
  LookupArgs a;
  a.table = table;
  a.ids = d_ids;
  a.out = d_out;
  a.err = d_err_word;
  a.n_rows = n_rows;
  a.n_ids = n_ids;
  a.dim = dim;
  a.scale = scale;
  a.in_dtype = table_dtype;
  a.out_dtype = out_dtype;
  return status_of(launch_lookup(a, static_cast<hipStream_t>(hip_stream)));
}

static bool grad_sizes_ok(uint64_t n_rows, uint64_t n_ids, uint32_t dim) {
  return n_rows < 0xFFFFFFFFull && n_ids < IBP_MAX_TOKENS && dim <= IBP_MAX_COLS;
}

IBP_API uint64_t ibp_embedding_grad_workspace_bytes(uint64_t n_rows, uint64_t n_ids, uint32_t dim) {
  return grad_sizes_ok(n_rows, n_ids, dim) ? embed_grad_workspace(n_rows, n_ids, dim) : 0;
}

IBP_API int ibp_embedding_grad(const void *d_dout, int dout_dtype, const int64_t *d_ids, uint64_t n_ids,
                               uint64_t n_rows, uint32_t dim, float scale, int64_t padding_id, void *d_grad,
                               int grad_dtype, void *d_workspace, uint64_t workspace_bytes, uint32_t *d_err_word,
                               void *hip_stream) {
  if (!dtype_ok(dout_dtype) || !dtype_ok(grad_dtype) || padding_id < -1) return IBP_ERR_INVALID_ARG;
  if (!grad_sizes_ok(n_rows, n_ids, dim) || (n_rows == 0 && n_ids > 0)) return IBP_ERR_SIZE;
  uint64_t db, gb;
  if (!matrix_bytes(n_ids, dim, dtype_size(dout_dtype), &db) || !matrix_bytes(n_rows, dim, dtype_size(grad_dtype), &gb))
    return IBP_ERR_SIZE;
  if (n_rows == 0 || dim == 0) return IBP_OK;
  const uint64_t wb = embed_grad_workspace(n_rows, n_ids, dim);
  if (workspace_bytes < wb) return IBP_ERR_CAPACITY;
  if (!d_grad || !d_workspace || (n_ids && (!d_dout || !d_ids))) return IBP_ERR_INVALID_ARG;
  if (!aligned(d_dout, dtype_size(dout_dtype)) || !aligned(d_ids, 8) || !aligned(d_grad, dtype_size(grad_dtype)) ||
      !aligned(d_workspace, 16) || !aligned(d_err_word, 4))
    return IBP_ERR_INVALID_ARG;
  Views see;
  if (!see(d_dout, db) || !see(d_ids, 8 * n_ids) || !see(d_grad, gb) || !see(d_workspace, wb) ||
      !see(d_err_word, d_err_word ? 4 : 0))
    return IBP_ERR_INVALID_ARG;
  EmbedGradArgs a;
  a.dout = d_dout;
  a.ids = d_ids;
  a.grad = d_grad;
  a.err = d_err_word;
  a.ws = static_cast<uint8_t *>(d_workspace);
  a.n_rows = n_rows;
  a.n_ids = n_ids;
  a.padding_id = padding_id;
  a.dim = dim;
  a.scale = scale;
  a.in_dtype = dout_dtype;
  a.out_dtype = grad_dtype;
  return status_of(launch_embed_grad(a, static_cast<hipStream_t>(hip_stream)));
}

IBP_API uint64_t ibp_mx_codes_pitch(uint64_t cols, uint32_t format) {
  if (format > IBP_MX_E2M1 || cols > IBP_MAX_COLS) return 0;
  return mx_code_pitch(cols, format == IBP_MX_E4M3);
}

IBP_API uint64_t ibp_mx_scales_pitch(uint64_t cols) { return cols > IBP_MAX_COLS ? 0 : mx_scale_pitch(cols); }

// Field checks of a packed tensor, before any HIP call.
static int mx_check(const ibp_mx_t *t) {
  if (!t || t->format > IBP_MX_E2M1 || t->reserved) return IBP_ERR_INVALID_ARG;
  uint64_t b;
  if (t->cols > IBP_MAX_COLS || !mul_ok(t->rows, mx_code_pitch(t->cols, true), &b)) return IBP_ERR_SIZE;
  if (!aligned(t->codes, 16) || !aligned(t->scales, 4)) return IBP_ERR_INVALID_ARG;
  if (t->rows && t->cols && (!t->codes || !t->scales)) return IBP_ERR_INVALID_ARG;
  return IBP_OK;
}

// The tensor's device pointers, checked against their allocations.
static bool mx_view(Views &see, const ibp_mx_t *t, uint8_t **codes, uint8_t **scales) {
  *codes = t->codes;
  *scales = t->scales;
  return see(*codes, t->rows * mx_code_pitch(t->cols, t->format == IBP_MX_E4M3)) &&
         see(*scales, t->rows * mx_scale_pitch(t->cols));
}

static void mx_fill(MxArgs *a, const ibp_mx_t *t, int dtype) {
  memset(a, 0, sizeof(*a));
  a->rows = t->rows;
  a->cols = (uint32_t)t->cols;
  a->e4m3 = t->format == IBP_MX_E4M3;
  a->dtype = dtype;
}

IBP_API int ibp_mx_pack(const void *d_in, int dtype, const ibp_mx_t *out, void *hip_stream) {
  if (!dtype_ok(dtype)) return IBP_ERR_INVALID_ARG;
  if (const int rc = mx_check(out)) return rc;
  uint64_t b;
  if (!matrix_bytes(out->rows, out->cols, dtype_size(dtype), &b)) return IBP_ERR_SIZE;
  if (b == 0) return IBP_OK;
  if (!d_in || !aligned(d_in, dtype_size(dtype))) return IBP_ERR_INVALID_ARG;
  MxArgs a;
  mx_fill(&a, out, dtype);
  Views see;
  if (!see(d_in, b) || !mx_view(see, out, &a.codes, &a.scales)) return IBP_ERR_INVALID_ARG;
  a.in = d_in;
  return status_of(launch_mx_pack(a, static_cast<hipStream_t>(hip_stream)));
}

IBP_API int ibp_mx_unpack(const ibp_mx_t *in, void *d_out, int dtype, void *hip_stream) {
  if (!dtype_ok(dtype)) return IBP_ERR_INVALID_ARG;
  if (const int rc = mx_check(in)) return rc;
  uint64_t b;
  if (!matrix_bytes(in->rows, in->cols, dtype_size(dtype), &b)) return IBP_ERR_SIZE;
  if (b == 0) return IBP_OK;
  if (!d_out || !aligned(d_out, dtype_size(dtype))) return IBP_ERR_INVALID_ARG;
  MxArgs a;
  mx_fill(&a, in, dtype);
  Views see;
  if (!see(d_out, b) || !mx_view(see, in, &a.codes, &a.scales)) return IBP_ERR_INVALID_ARG;
  a.out = d_out;
  return status_of(launch_mx_unpack(a, static_cast<hipStream_t>(hip_stream)));
}

// Checks shared by the gated activation's two directions: two e4m3 checkpoints of one
// shape, three plain tensors of it.
static int gated_check(const void *x, const void *y, const void *z, int dtype, const ibp_mx_t *gate8,
                       const ibp_mx_t *up8, uint64_t *bytes) {
  if (!dtype_ok(dtype)) return IBP_ERR_INVALID_ARG;
  if (const int rc = mx_check(gate8)) return rc;
  if (const int rc = mx_check(up8)) return rc;
  if (gate8->format != IBP_MX_E4M3 || up8->format != IBP_MX_E4M3) return IBP_ERR_INVALID_ARG;
  if (gate8->rows != up8->rows || gate8->cols != up8->cols) return IBP_ERR_SIZE;
  if (!matrix_bytes(gate8->rows, gate8->cols, dtype_size(dtype), bytes)) return IBP_ERR_SIZE;
  if (*bytes == 0) return IBP_OK;
  for (const void *p : {x, y, z})
    if (!p || !aligned(p, dtype_size(dtype))) return IBP_ERR_INVALID_ARG;
  return IBP_OK;
}

static bool overlap(const Range &x, const Range &y) {
  return x.bytes && y.bytes && (uintptr_t)x.p < (uintptr_t)y.p + y.bytes && (uintptr_t)y.p < (uintptr_t)x.p + x.bytes;
}

// Whether outputs lie apart from each other and from the inputs.  The first plain_outs and
// plain_ins of them are plain tensors: such an output may be such an input itself where what
// a lane writes is read by that lane alone, or before by its own wavefront: the last lane of a
// row reads the row's last eight elements, some of them its neighbour's, and a row of up to
// 512 elements belongs to one wavefront.
static bool apart(std::initializer_list<Range> outs, uint32_t plain_outs, std::initializer_list<Range> ins,
                  uint32_t plain_ins, uint64_t cols) {
  const bool in_place = cols % 8 == 0 || cols <= 512;
  for (const Range *o = outs.begin(); o != outs.end(); ++o) {
    for (const Range *q = o + 1; q != outs.end(); ++q)
      if (overlap(*o, *q)) return false;
    for (const Range *i = ins.begin(); i != ins.end(); ++i) {
      const bool itself = o->p == i->p && o < outs.begin() + plain_outs && i < ins.begin() + plain_ins;
      if (overlap(*o, *i) && !(itself && in_place)) return false;
    }
  }
  return true;
}

static Range codes_range(const ibp_mx_t *t) { return {t->codes, t->rows * mx_code_pitch(t->cols, t->format == IBP_MX_E4M3)}; }
static Range scales_range(const ibp_mx_t *t) { return {t->scales, t->rows * mx_scale_pitch(t->cols)}; }

IBP_API int ibp_mx_swiglu(const void *d_gate, const void *d_up, int dtype, void *d_h, const ibp_mx_t *gate8,
                          const ibp_mx_t *up8, void *hip_stream) {
  uint64_t b = 0;
  if (const int rc = gated_check(d_gate, d_up, d_h, dtype, gate8, up8, &b)) return rc;
  if (b == 0) return IBP_OK;
  if (!apart({{d_h, b}, codes_range(gate8), scales_range(gate8), codes_range(up8), scales_range(up8)}, 1,
             {{d_gate, b}, {d_up, b}}, 2, gate8->cols))
    return IBP_ERR_INVALID_ARG;
  MxArgs a;
  mx_fill(&a, gate8, dtype);
  Views see;
  if (!see(d_gate, b) || !see(d_up, b) || !see(d_h, b) || !mx_view(see, gate8, &a.codes, &a.scales) ||
      !mx_view(see, up8, &a.codes2, &a.scales2))
    return IBP_ERR_INVALID_ARG;
  a.in = d_gate;
  a.in2 = d_up;
  a.out = d_h;
  return status_of(launch_mx_swiglu(a, static_cast<hipStream_t>(hip_stream)));
}

IBP_API int ibp_mx_swiglu_backward(const void *d_dh, int dtype, const ibp_mx_t *gate8, const ibp_mx_t *up8,
                                   void *d_dgate, void *d_dup, void *hip_stream) {
  uint64_t b = 0;
  if (const int rc = gated_check(d_dh, d_dgate, d_dup, dtype, gate8, up8, &b)) return rc;
  if (b == 0) return IBP_OK;
  if (!apart({{d_dgate, b}, {d_dup, b}}, 2,
             {{d_dh, b}, codes_range(gate8), scales_range(gate8), codes_range(up8), scales_range(up8)}, 1, gate8->cols))
    return IBP_ERR_INVALID_ARG;
  MxArgs a;
  mx_fill(&a, gate8, dtype);
  Views see;
  if (!see(d_dh, b) || !see(d_dgate, b) || !see(d_dup, b) || !mx_view(see, gate8, &a.codes, &a.scales) ||
      !mx_view(see, up8, &a.codes2, &a.scales2))
    return IBP_ERR_INVALID_ARG;
  a.in2 = d_dh;
  a.out = d_dgate;
  a.out2 = d_dup;
  return status_of(launch_mx_swiglu_backward(a, static_cast<hipStream_t>(hip_stream)));
}

// Rows of a product: the launch grids and 32-bit row numbers hold up to 2^30.
static bool product_rows_ok(uint64_t n) { return n <= IBP_MAX_COLS; }

IBP_API uint64_t ibp_mx_matmul_workspace_bytes(uint64_t m, uint64_t n, uint64_t k, uint32_t a_format) {
  if (!product_rows_ok(m) || !product_rows_ok(n) || k > IBP_MAX_COLS || a_format > IBP_MX_E2M1) return 0;
  return m && n ? mx_matmul_workspace(m, n, (uint32_t)k) : 0;
}

IBP_API uint64_t ibp_mx_linear_wgrad_workspace_bytes(uint64_t tokens, uint64_t outs, uint64_t ins, int dy_dtype) {
  if (!product_rows_ok(outs) || ins > IBP_MAX_COLS || !dtype_ok(dy_dtype)) return 0;
  return outs && ins ? mx_wgrad_workspace(tokens, (uint32_t)outs, (uint32_t)ins, dy_dtype) : 0;
}

IBP_API int ibp_mx_matmul(const ibp_mx_t *a, const ibp_mx_t *b, void *d_y, int dtype, void *d_workspace,
                          uint64_t workspace_bytes, void *hip_stream) {
  if (!dtype_ok(dtype)) return IBP_ERR_INVALID_ARG;
  if (const int rc = mx_check(a)) return rc;
  if (const int rc = mx_check(b)) return rc;
  if (b->format != IBP_MX_E2M1) return IBP_ERR_INVALID_ARG;
  uint64_t yb;
  if (a->cols != b->cols || !product_rows_ok(a->rows) || !product_rows_ok(b->rows) ||
      !matrix_bytes(a->rows, b->rows, dtype_size(dtype), &yb))
    return IBP_ERR_SIZE;
  if (yb == 0) return IBP_OK;
  const uint64_t wb = mx_matmul_workspace(a->rows, b->rows, (uint32_t)a->cols);
  if (workspace_bytes < wb) return IBP_ERR_CAPACITY;
  if (!d_y || !aligned(d_y, dtype_size(dtype)) || (wb && !d_workspace) || !aligned(d_workspace, 16))
    return IBP_ERR_INVALID_ARG;
  uint8_t *ac, *as, *bc, *bs;
  Views see;
  if (!see(d_y, yb) || !mx_view(see, a, &ac, &as) || !mx_view(see, b, &bc, &bs) || !see(d_workspace, wb))
    return IBP_ERR_INVALID_ARG;
  MxMatmulArgs p;
  p.a_codes = ac;
  p.a_scales = as;
  p.b_codes = bc;
  p.b_scales = bs;
  p.y = d_y;
  p.ws = static_cast<float *>(d_workspace);
  p.M = a->rows;
  p.N = b->rows;
  p.K = (uint32_t)a->cols;
  p.a_e4m3 = a->format == IBP_MX_E4M3;
  p.dtype = dtype;
  p.offsets = nullptr;
  p.experts = 0;
  p.err = nullptr;
  return status_of(launch_mx_matmul(p, static_cast<hipStream_t>(hip_stream)));
}

IBP_API int ibp_mx_linear_wgrad(const void *d_dy, int dy_dtype, uint64_t outs, const ibp_mx_t *x8, void *d_dw,
                                int dw_dtype, void *d_workspace, uint64_t workspace_bytes, void *hip_stream) {
  if (!dtype_ok(dy_dtype) || !dtype_ok(dw_dtype)) return IBP_ERR_INVALID_ARG;
  if (const int rc = mx_check(x8)) return rc;
  if (x8->format != IBP_MX_E4M3) return IBP_ERR_INVALID_ARG;
  uint64_t yb, wgb;
  if (!product_rows_ok(outs) || !matrix_bytes(x8->rows, outs, dtype_size(dy_dtype), &yb) ||
      !matrix_bytes(outs, x8->cols, dtype_size(dw_dtype), &wgb))
    return IBP_ERR_SIZE;
  if (wgb == 0) return IBP_OK;
  const uint64_t wb = mx_wgrad_workspace(x8->rows, (uint32_t)outs, (uint32_t)x8->cols, dy_dtype);
  if (workspace_bytes < wb) return IBP_ERR_CAPACITY;
  if (!d_dw || !aligned(d_dw, dtype_size(dw_dtype)) || (yb && !d_dy) || !aligned(d_dy, dtype_size(dy_dtype)) || (wb && !d_workspace) ||
      !aligned(d_workspace, 16))
    return IBP_ERR_INVALID_ARG;
  uint8_t *xc, *xs;
  Views see;
  if (!see(d_dy, yb) || !mx_view(see, x8, &xc, &xs) || !see(d_dw, wgb) || !see(d_workspace, wb))
    return IBP_ERR_INVALID_ARG;
  MxWgradArgs p;
  p.dy = d_dy;
  p.x_codes = xc;
  p.x_scales = xs;
  p.dw = d_dw;
  p.ws = static_cast<float *>(d_workspace);
  p.T = x8->rows;
  p.N = (uint32_t)outs;
  p.K = (uint32_t)x8->cols;
  p.dy_dtype = dy_dtype;
  p.dtype = dw_dtype;
  p.offsets = nullptr;
  p.experts = 0;
  p.err = nullptr;
  return status_of(launch_mx_wgrad(p, static_cast<hipStream_t>(hip_stream)));
}

// ------------------------------------------------------------------ 8-bit integer rows

IBP_API uint64_t ibp_i8_codes_pitch(uint64_t cols) { return cols > IBP_MAX_COLS ? 0 : i8_pitch(cols); }

// Field checks of a tensor of 8-bit integer rows, before any HIP call.
static int i8_check(const ibp_i8_t *t) {
  if (!t) return IBP_ERR_INVALID_ARG;
  uint64_t b;
  if (t->cols > IBP_MAX_COLS || !matrix_bytes(t->rows, i8_pitch(t->cols), 1, &b) || !mul_ok(t->rows, 4, &b)) return IBP_ERR_SIZE;
  if (!aligned(t->codes, 16) || !aligned(t->scales, 4)) return IBP_ERR_INVALID_ARG;
  if (t->rows && (!t->scales || (t->cols && !t->codes))) return IBP_ERR_INVALID_ARG;
  return IBP_OK;
}

static Range codes_range(const ibp_i8_t *t) { return {t->codes, t->rows * i8_pitch(t->cols)}; }
static Range scales_range(const ibp_i8_t *t) { return {t->scales, t->rows * 4}; }

static bool i8_view(Views &see, const ibp_i8_t *t, int8_t **codes, float **scales) {
  *codes = t->codes;
  *scales = t->scales;
  return see(*codes, codes_range(t).bytes) && see(*scales, scales_range(t).bytes);
}

IBP_API int ibp_i8_pack(const void *d_in, int dtype, const ibp_i8_t *out, void *hip_stream) {
  if (!dtype_ok(dtype)) return IBP_ERR_INVALID_ARG;
  if (const int rc = i8_check(out)) return rc;
  uint64_t b;
  if (!matrix_bytes(out->rows, out->cols, dtype_size(dtype), &b)) return IBP_ERR_SIZE;
  if (out->rows == 0) return IBP_OK;
  if ((b && !d_in) || !aligned(d_in, dtype_size(dtype))) return IBP_ERR_INVALID_ARG;
  if (!apart({codes_range(out), scales_range(out)}, 0, {{d_in, b}}, 0, 0)) return IBP_ERR_INVALID_ARG;
  I8Args a;
  Views see;
  if (!see(d_in, b) || !i8_view(see, out, &a.codes, &a.scales)) return IBP_ERR_INVALID_ARG;
  a.in = d_in;
  a.out = nullptr;
  a.rows = out->rows;
  a.cols = (uint32_t)out->cols;
  a.dtype = dtype;
  return status_of(launch_i8_pack(a, static_cast<hipStream_t>(hip_stream)));
}

IBP_API int ibp_i8_unpack(const ibp_i8_t *in, void *d_out, int dtype, void *hip_stream) {
  if (!dtype_ok(dtype)) return IBP_ERR_INVALID_ARG;
  if (const int rc = i8_check(in)) return rc;
  uint64_t b;
  if (!matrix_bytes(in->rows, in->cols, dtype_size(dtype), &b)) return IBP_ERR_SIZE;
  if (b == 0) return IBP_OK;
  if (!d_out || !aligned(d_out, dtype_size(dtype))) return IBP_ERR_INVALID_ARG;
  if (!apart({{d_out, b}}, 0, {codes_range(in), scales_range(in)}, 0, 0)) return IBP_ERR_INVALID_ARG;
  I8Args a;
  Views see;
  if (!see(d_out, b) || !i8_view(see, in, &a.codes, &a.scales)) return IBP_ERR_INVALID_ARG;
  a.in = nullptr;
  a.out = d_out;
  a.rows = in->rows;
  a.cols = (uint32_t)in->cols;
  a.dtype = dtype;
  return status_of(launch_i8_unpack(a, static_cast<hipStream_t>(hip_stream)));
}

IBP_API uint64_t ibp_i8_matmul_workspace_bytes(uint64_t m, uint64_t n, uint64_t k) {
  if (!product_rows_ok(m) || !product_rows_ok(n) || k > IBP_I8_MAX_DEPTH) return 0;
  return m && n ? i8_matmul_workspace(m, n, (uint32_t)k) : 0;
}

IBP_API int ibp_i8_matmul(const ibp_i8_t *a, const ibp_i8_t *b, void *d_y, int dtype, void *d_workspace,
                          uint64_t workspace_bytes, void *hip_stream) {
  if (!dtype_ok(dtype)) return IBP_ERR_INVALID_ARG;
  if (const int rc = i8_check(a)) return rc;
  if (const int rc = i8_check(b)) return rc;
  uint64_t yb;
  if (a->cols != b->cols || a->cols > IBP_I8_MAX_DEPTH || !product_rows_ok(a->rows) || !product_rows_ok(b->rows) ||
      !matrix_bytes(a->rows, b->rows, dtype_size(dtype), &yb))
    return IBP_ERR_SIZE;
  if (yb == 0) return IBP_OK;
  const uint64_t wb = i8_matmul_workspace(a->rows, b->rows, (uint32_t)a->cols);
  if (workspace_bytes < wb) return IBP_ERR_CAPACITY;
  if (!d_y || !aligned(d_y, dtype_size(dtype)) || (wb && !d_workspace) || !aligned(d_workspace, 16))
    return IBP_ERR_INVALID_ARG;
  if (!apart({{d_y, yb}, {d_workspace, wb}}, 0, {codes_range(a), scales_range(a), codes_range(b), scales_range(b)}, 0, 0))
    return IBP_ERR_INVALID_ARG;
  int8_t *ac, *bc;
  float *as, *bs;
  Views see;
  if (!see(d_y, yb) || !i8_view(see, a, &ac, &as) || !i8_view(see, b, &bc, &bs) || !see(d_workspace, wb)) return IBP_ERR_INVALID_ARG;
  I8MatmulArgs p;
  p.a_codes = reinterpret_cast<const uint8_t *>(ac);
  p.b_codes = reinterpret_cast<const uint8_t *>(bc);
  p.a_scales = as;
  p.b_scales = bs;
  p.y = d_y;
  p.ws = static_cast<int32_t *>(d_workspace);
  p.M = a->rows;
  p.N = b->rows;
  p.K = (uint32_t)a->cols;
  p.dtype = dtype;
  return status_of(launch_i8_matmul(p, static_cast<hipStream_t>(hip_stream)));
}

// ------------------------------------------------------------------ experts

static bool experts_ok(uint64_t n) { return n >= 1 && n <= IBP_MAX_EXPERTS; }

IBP_API uint64_t ibp_expert_order_workspace_bytes(uint64_t n_ids, uint64_t n_experts) {
  return n_ids < IBP_MAX_TOKENS && experts_ok(n_experts) ? expert_order_workspace(n_ids, (uint32_t)n_experts) : 0;
}

IBP_API int ibp_expert_order(const int64_t *d_ids, uint64_t n_ids, uint64_t n_experts, int64_t *d_order,
                             int64_t *d_offsets, void *d_workspace, uint64_t workspace_bytes, uint32_t *d_err_word,
                             void *hip_stream) {
  if (n_ids >= IBP_MAX_TOKENS || !experts_ok(n_experts)) return IBP_ERR_SIZE;
  const uint64_t wb = expert_order_workspace(n_ids, (uint32_t)n_experts), ib = n_ids * 8, ob = (n_experts + 1) * 8;
  if (workspace_bytes < wb) return IBP_ERR_CAPACITY;
  if (!d_offsets || (n_ids && (!d_ids || !d_order)) || (wb && !d_workspace)) return IBP_ERR_INVALID_ARG;
  if (!aligned(d_ids, 8) || !aligned(d_order, 8) || !aligned(d_offsets, 8) || !aligned(d_workspace, 16) || !aligned(d_err_word, 4))
    return IBP_ERR_INVALID_ARG;
  if (!apart({{d_order, ib}, {d_offsets, ob}, {d_workspace, wb}}, 0, {{d_ids, ib}}, 0, 0)) return IBP_ERR_INVALID_ARG;
  Views see;
  if (!see(d_ids, ib) || !see(d_order, ib) || !see(d_offsets, ob) || !see(d_workspace, wb) || !see(d_err_word, d_err_word ? 4 : 0))
    return IBP_ERR_INVALID_ARG;
  ExpertOrderArgs a;
  a.ids = d_ids;
  a.order = d_order;
  a.offsets = d_offsets;
  a.counts = static_cast<uint32_t *>(d_workspace);
  a.err = d_err_word;
  a.n = n_ids;
  a.experts = (uint32_t)n_experts;
  return status_of(launch_expert_order(a, static_cast<hipStream_t>(hip_stream)));
}

IBP_API int ibp_mx_grouped_matmul(const ibp_mx_t *a, const ibp_mx_t *b, const int64_t *d_offsets, uint64_t n_experts,
                                  void *d_y, int dtype, uint32_t *d_err_word, void *hip_stream) {
  if (!dtype_ok(dtype)) return IBP_ERR_INVALID_ARG;
  if (const int rc = mx_check(a)) return rc;
  if (const int rc = mx_check(b)) return rc;
  if (b->format != IBP_MX_E2M1) return IBP_ERR_INVALID_ARG;
  if (!experts_ok(n_experts) || b->rows % n_experts) return IBP_ERR_SIZE;
  const uint64_t N = b->rows / n_experts;
  uint64_t yb;
  if (a->cols != b->cols || !product_rows_ok(a->rows) || !product_rows_ok(N) ||
      !matrix_bytes(a->rows, N, dtype_size(dtype), &yb))
    return IBP_ERR_SIZE;
  if (yb == 0) return IBP_OK;
  const uint64_t ob = (n_experts + 1) * 8;
  if (!d_y || !aligned(d_y, dtype_size(dtype)) || !d_offsets || !aligned(d_offsets, 8) || !aligned(d_err_word, 4))
    return IBP_ERR_INVALID_ARG;
  if (!apart({{d_y, yb}}, 0,
             {codes_range(a), scales_range(a), codes_range(b), scales_range(b), {d_offsets, ob}}, 0, 0))
    return IBP_ERR_INVALID_ARG;
  uint8_t *ac, *as, *bc, *bs;
  Views see;
  if (!see(d_y, yb) || !mx_view(see, a, &ac, &as) || !mx_view(see, b, &bc, &bs) || !see(d_offsets, ob) ||
      !see(d_err_word, d_err_word ? 4 : 0))
    return IBP_ERR_INVALID_ARG;
  MxMatmulArgs p;
  p.a_codes = ac;
  p.a_scales = as;
  p.b_codes = bc;
  p.b_scales = bs;
  p.y = d_y;
  p.ws = nullptr;
  p.M = a->rows;
  p.N = N;
  p.K = (uint32_t)a->cols;
  p.a_e4m3 = a->format == IBP_MX_E4M3;
  p.dtype = dtype;
  p.offsets = d_offsets;
  p.experts = (uint32_t)n_experts;
  p.err = d_err_word;
  return status_of(launch_mx_grouped_matmul(p, static_cast<hipStream_t>(hip_stream)));
}

static bool grouped_sizes_ok(uint64_t tokens, uint64_t n_experts, uint64_t outs, uint64_t ins) {
  return tokens < IBP_MAX_TOKENS && experts_ok(n_experts) && product_rows_ok(outs) && ins <= IBP_MAX_COLS;
}

IBP_API uint64_t ibp_mx_grouped_wgrad_workspace_bytes(uint64_t tokens, uint64_t n_experts, uint64_t outs, uint64_t ins,
                                                      int dy_dtype, const void *d_dy) {
  if (!grouped_sizes_ok(tokens, n_experts, outs, ins) || !dtype_ok(dy_dtype)) return 0;
  return outs && ins ? mx_grouped_wgrad_workspace(tokens, (uint32_t)n_experts, (uint32_t)outs, (uint32_t)ins, dy_dtype,
                                                   d_dy && aligned(d_dy, 16))
                      : 0;
}

IBP_API int ibp_mx_grouped_wgrad(const void *d_dy, int dy_dtype, uint64_t outs, const ibp_mx_t *x8,
                                 const int64_t *d_offsets, uint64_t n_experts, void *d_dw, int dw_dtype,
                                 void *d_workspace, uint64_t workspace_bytes, uint32_t *d_err_word, void *hip_stream) {
  if (!dtype_ok(dy_dtype) || !dtype_ok(dw_dtype)) return IBP_ERR_INVALID_ARG;
  if (const int rc = mx_check(x8)) return rc;
  if (x8->format != IBP_MX_E4M3) return IBP_ERR_INVALID_ARG;
  uint64_t yb, wgb;
  if (!grouped_sizes_ok(x8->rows, n_experts, outs, x8->cols) || !matrix_bytes(x8->rows, outs, dtype_size(dy_dtype), &yb) ||
      !matrix_bytes(n_experts * outs, x8->cols, dtype_size(dw_dtype), &wgb))
    return IBP_ERR_SIZE;
  if (wgb == 0) return IBP_OK;
  const uint64_t wb = mx_grouped_wgrad_workspace(x8->rows, (uint32_t)n_experts, (uint32_t)outs, (uint32_t)x8->cols,
                                                 dy_dtype, aligned(d_dy, 16));
  const uint64_t ob = (n_experts + 1) * 8;
  if (workspace_bytes < wb) return IBP_ERR_CAPACITY;
  if (!d_dw || !aligned(d_dw, dtype_size(dw_dtype)) || (yb && !d_dy) || !aligned(d_dy, dtype_size(dy_dtype)) ||
      !d_offsets || !aligned(d_offsets, 8) || (wb && !d_workspace) || !aligned(d_workspace, 16) || !aligned(d_err_word, 4))
    return IBP_ERR_INVALID_ARG;
  if (!apart({{d_dw, wgb}, {d_workspace, wb}}, 0, {{d_dy, yb}, codes_range(x8), scales_range(x8), {d_offsets, ob}}, 0, 0))
    return IBP_ERR_INVALID_ARG;
  uint8_t *xc, *xs;
  Views see;
  if (!see(d_dy, yb) || !mx_view(see, x8, &xc, &xs) || !see(d_dw, wgb) || !see(d_offsets, ob) || !see(d_workspace, wb) ||
      !see(d_err_word, d_err_word ? 4 : 0))
    return IBP_ERR_INVALID_ARG;
  MxWgradArgs p;
  p.dy = d_dy;
  p.x_codes = xc;
  p.x_scales = xs;
  p.dw = d_dw;
  p.ws = static_cast<float *>(d_workspace);
  p.T = x8->rows;
  p.N = (uint32_t)outs;
  p.K = (uint32_t)x8->cols;
  p.dy_dtype = dy_dtype;
  p.dtype = dw_dtype;
  p.offsets = d_offsets;
  p.experts = (uint32_t)n_experts;
  p.err = d_err_word;
  return status_of(launch_mx_grouped_wgrad(p, static_cast<hipStream_t>(hip_stream)));
}

}  // extern "C"
