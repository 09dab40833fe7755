// ibp_ops.h -- arguments and launchers of the language-model operators, shared by the
// host entry points and the kernels.  Not part of the public ABI (that is include/ibp.h).
#pragma once

#include "ibp_internal.h"

namespace ibp {

// Embedding lookup and gradient.  Dtypes are IBP_F32 / IBP_F16 / IBP_BF16.
struct LookupArgs {
  const void *table;   // n_rows x dim (device or pinned host memory)
  const int64_t *ids;
  void *out;           // n_ids x dim
  uint32_t *err;       // optional
  uint64_t n_rows;
  uint64_t n_ids;
  uint32_t dim;
  float scale;
  int in_dtype;
  int out_dtype;
};

struct EmbedGradArgs {
  const void *dout;    // n_ids x dim
  const int64_t *ids;
  void *grad;          // n_rows x dim
  uint32_t *err;       // optional
  uint8_t *ws;         // embed_grad_workspace(...) bytes, aligned to 16
  uint64_t n_rows;
  uint64_t n_ids;      // < 2^31
  int64_t padding_id;  // this id takes no part; -1 for none
  uint32_t dim;
  float scale;
  int in_dtype;
  int out_dtype;
};
uint64_t embed_grad_workspace(uint64_t n_rows, uint64_t n_ids, uint32_t dim);

// Microscaled tensors: blocks of kMxBlock elements along a row.
constexpr uint32_t kMxBlock = 32;
__host__ __device__ constexpr uint64_t mx_blocks(uint64_t cols) { return (cols + kMxBlock - 1) / kMxBlock; }
__host__ __device__ constexpr uint64_t mx_scale_pitch(uint64_t cols) { return (mx_blocks(cols) + 3) / 4 * 4; }
__host__ __device__ constexpr uint64_t mx_code_pitch(uint64_t cols, bool e4m3) { return mx_blocks(cols) * (e4m3 ? 32 : 16); }

struct MxArgs {
  const void *in;      // pack: rows x cols; gated forward: gate
  const void *in2;     // gated forward: up; gated backward: dh
  void *out;           // unpack: rows x cols; gated forward: h; gated backward: dgate
  void *out2;          // gated backward: dup
  uint8_t *codes;
  uint8_t *scales;
  uint8_t *codes2;     // gated: the checkpoint of up
  uint8_t *scales2;
  uint64_t rows;
  uint32_t cols;
  bool e4m3;           // else e2m1
  int dtype;
};

struct MxMatmulArgs {
  const uint8_t *a_codes, *a_scales;  // M rows of K
  const uint8_t *b_codes, *b_scales;  // N rows of K, e2m1
  void *y;                            // M x N
  float *ws;                          // split partial sums, or null
  uint64_t M, N;
  uint32_t K;
  bool a_e4m3;
  int dtype;
};
uint64_t mx_matmul_workspace(uint64_t M, uint64_t N, uint32_t K);

struct MxWgradArgs {
  const void *dy;                     // T x N
  const uint8_t *x_codes, *x_scales;  // T rows of K, e4m3
  void *dw;                           // N x K
  float *ws;
  uint64_t T;
  uint32_t N, K;
  int dy_dtype;
  int dtype;
  uint32_t dy_pitch;  // set by the launch: elements from one row of dy to the next
};
uint64_t mx_wgrad_workspace(uint64_t T, uint32_t N, uint32_t K, int dy_dtype);

// Launchers.  Each returns the hipError_t of its launch(es).
hipError_t launch_lookup(const LookupArgs &a, hipStream_t s);  // ibp_embed.hip
hipError_t launch_embed_grad(const EmbedGradArgs &a, hipStream_t s);
hipError_t launch_mx_pack(const MxArgs &a, hipStream_t s);  // ibp_mx.hip
hipError_t launch_mx_unpack(const MxArgs &a, hipStream_t s);
hipError_t launch_mx_swiglu(const MxArgs &a, hipStream_t s);
hipError_t launch_mx_swiglu_backward(const MxArgs &a, hipStream_t s);
hipError_t launch_mx_matmul(const MxMatmulArgs &a, hipStream_t s);  // ibp_mx_matmul.hip
hipError_t launch_mx_wgrad(const MxWgradArgs &a, hipStream_t s);    // ibp_mx_wgrad.hip

}  // namespace ibp
