// One state space scan over prompts, already validated: what the entry points
// (ssm.cu) hand to the kernels.
#pragma once

#include "gdn_internal.h"

namespace gdn {

// Segments that a caller sets, and those on the tensor cores, are whole multiples of this many
// tokens; on CUDA cores the library's choice may be of half of it.
constexpr int SSM_UNIT = 128;
// The segment length that leaves every sequence whole.
constexpr int SSM_WHOLE = 0x7fffff80;

struct SsmParams {
  const void *x, *z, *Bm, *Cm, *dt;
  const float *A_log, *D, *dt_bias;
  const float *h0;
  float *ht;
  void *y;
  const int32_t *cu;
  int *err;
  int64_t xs, xb, zs, zb, bs, bb, cs, cb, dts, dtb, ys, yb;  // token and batch strides
  int B, T, H, Hg, K, V, N;
  int dt_f32, softplus, y_f32;
  // Sequences are cut into segments of `seg` tokens (the last one shorter; an
  // empty sequence is one empty segment).  `items` bounds their number.
  int seg, items;
  // Only when a sequence can have more than one segment: each segment's last
  // state from zero [items][H][V][K] and the logarithm of its decay [items][H].
  float *seg_state, *seg_decay;
};

// The scan on the tensor cores: whether it serves p, and its launch.
bool ssm_tc_supported(const SsmParams &p, bool bf16);
cudaError_t launch_ssm_tc(const SsmParams &p, cudaStream_t stream);
// The scan in float32 on the CUDA cores: any type and size.
cudaError_t launch_ssm_simt(const SsmParams &p, bool bf16, cudaStream_t stream);

}  // namespace gdn
