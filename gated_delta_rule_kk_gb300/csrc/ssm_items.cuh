// Which tokens a segment of the state space scan covers (device code shared by
// its kernels).
#pragma once

#include "gdn_common.cuh"
#include "ssm.h"

namespace gdn {

struct SsmItem {
  int n, b;         // sequence and batch row
  int bos, eos;     // the sequence's tokens
  int lo, hi;       // the segment's tokens
  int first;        // index of the sequence's first segment
  bool last;        // whether it is the sequence's last segment
};

// Segment `item` (offsets checked; every thread of the warp takes part and
// gets the same answer), or n = -1 past the last one.  Sequence n holds
// max(1, ceil(len / seg)) segments, numbered sequence after sequence.
__device__ __forceinline__ SsmItem ssm_item(const SsmParams &p, int item) {
  SsmItem r;
  auto segments = [&](int len) { return len > p.seg ? (len - 1) / p.seg + 1 : 1; };
  r.n = -1;
  if (p.cu == nullptr) {
    const int each = segments(p.T);
    if (item >= each * p.N) return r;
    r.n = r.b = item / each;
    r.first = r.n * each;
    r.bos = 0;
    r.eos = p.T;
  } else {
    const int lane = threadIdx.x & 31;
    int before = 0;
    for (int base = 0; base < p.N; base += 32) {
      const int n = base + lane;
      const int len = n < p.N ? p.cu[n + 1] - p.cu[n] : 0;
      const int own = n < p.N ? segments(len) : 0;
      int sum = own;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const int v = __shfl_up_sync(~0u, sum, o);
        if (lane >= o) sum += v;
      }
      const unsigned past = __ballot_sync(~0u, before + sum > item);
      if (past) {
        const int l = __ffs(past) - 1;
        r.n = base + l;
        r.first = before + __shfl_sync(~0u, sum - own, l);
        r.bos = p.cu[r.n];
        r.eos = p.cu[r.n + 1];
        break;
      }
      before += __shfl_sync(~0u, sum, 31);
    }
    if (r.n < 0) return r;
    r.b = 0;
  }
  r.lo = r.bos + (item - r.first) * p.seg;
  r.hi = r.eos - r.lo > p.seg ? r.lo + p.seg : r.eos;
  r.last = r.hi == r.eos;
  return r;
}

// dt at element `at`, and the step size from dt with its bias.
template <typename Params>
__device__ __forceinline__ float ssm_dt(const Params &p, int64_t at) {
  return p.dt_f32 ? static_cast<const float *>(p.dt)[at]
                  : to_f32(static_cast<const __nv_bfloat16 *>(p.dt)[at]);
}
template <typename Params>
__device__ __forceinline__ float ssm_softplus(const Params &p, float v) {
  return p.softplus ? softplus(v) : v;
}
// Step size of a token and head.
template <typename Params>
__device__ __forceinline__ float ssm_step(const Params &p, int64_t row, int h, float bias) {
  return ssm_softplus(p, ssm_dt(p, row + h) + bias);
}

}  // namespace gdn
