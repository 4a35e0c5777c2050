// The gated delta rule's gradient over chunks, between its entry point (delta_bwd.cu) and
// the kernels (delta_bwd_tc.cu on the tensor cores, delta_bwd_simt.cu on CUDA cores).
//
// Per chunk of 64 tokens, with G the running sum of the log-gates, h the state [K, V] at the
// chunk's start and D the gradient of the state at its end:
//   A_ij = beta_i k_i.k_j e^(G_i - G_j)  (i > j),   P_ij = scale q_i.k_j e^(G_i - G_j)  (i >= j)
//   T = (I + A)^-1,  r = beta (v - e^G k h),  n = T r,  h+ = e^(G_L) h + (k e^(G_L - G))^T n
// and back:
//   dn = P^T do + e^(G_L - G) k D,   dr = T^T dn,
//   D- = e^(G_L) D + (scale e^G q)^T do - (beta e^G k)^T dr,
//   dA = -dr n^T (i > j),   dP = do n^T (i >= j),
//   dq = scale e^G do h^T + (dP L) k,                      L_ij = e^(G_i - G_j), scale in dP L
//   dk = -beta e^G dr h^T + e^(G_L - G) n D^T + (dP L)^T q + (dA L beta + its transpose) k,
//   dv = beta dr,   dbeta = dr.v - e^G k.(dr h^T) + rowsum(dA k k^T L),
//   dG = rowsum(M) - colsum(M) + q.dq_h + k.dk_h - k.dk_s,   M = dA A + dP P,
//   dG_L += e^(G_L) <h, D> + sum k.dk_s,
// where dq_h, dk_h and dk_s are the terms with h and D; dg is dG summed from the chunk's end.
// (There k.dk_s is what the tokens before add up to, and M's diagonal cancels: neither is summed
// and taken off again, so that next to a gate that forgets, whose dg is as small as e^g, nothing
// of order one has to cancel.)
// (dA = -dr n^T holds as n solves (I + A) n = r: neither the gradient of T nor w = T beta e^G k
// is formed.)  Four launches (five with packed sequences): T and P of every chunk; the states forward; their gradients
// backward; everything else, every chunk by itself.
#pragma once

#include <cuda_runtime.h>
#include <stdint.h>

#include "gdn.h"

namespace gdn {

struct DeltaBwdParams {
  const void *q, *k, *v, *dout;
  const float *g, *beta, *h0, *dht;
  void *dq, *dk, *dv;
  float *dg, *dbeta, *dh0;
  const int32_t *cu;
  int *err;
  int B, T, H, Hg, K, V, N;
  int g_is_cumsum, v_first;
  float scale;
  int per_seq;                // chunks of a sequence (cu NULL)
  int64_t chunks;             // chunks at most
  // workspace
  int32_t *first;             // [N + 1] first chunk of every sequence (cu given)
  int32_t *order;             // [N] the sequences, longest first (about)
  int32_t *owner;             // [chunks] sequence of every chunk
  unsigned char *blocks;      // [chunks][H] of `block` bytes each
  int64_t block;
  float *scratch;             // of delta_bwd_tc_scratch() bytes, behind the blocks
};

// A chunk: its sequence, its place there, its first token and how many it has.
struct DeltaChunk {
  int n, i, len;
  int64_t token;
};

#ifdef __CUDACC__
// Launches a kernel that may begin while the one before it on the stream ends; it waits
// (griddepcontrol.wait) before it reads anything.
template <typename... P, typename... A>
cudaError_t launch_behind(void (*kernel)(P...), dim3 grid, int threads, int smem, cudaStream_t stream,
                          const A &...args) {
  cudaLaunchAttribute early{};
  early.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  early.val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = grid;
  cfg.blockDim = dim3(threads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = stream;
  cfg.attrs = &early;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kernel, args...);
}

// Chunk c; len 0 if there is none.
__device__ __forceinline__ DeltaChunk delta_chunk(const DeltaBwdParams &p, int64_t c) {
  DeltaChunk k{0, 0, 0, 0};
  if (p.cu == nullptr) {
    k.n = (int)(c / p.per_seq);
    k.i = (int)(c - (int64_t)k.n * p.per_seq);
    k.len = min(64, p.T - k.i * 64);
    k.token = (int64_t)k.n * p.T + k.i * 64;
    return k;
  }
  if (c >= p.first[p.N]) return k;
  k.n = p.owner[c];
  k.i = (int)(c - p.first[k.n]);
  const int lo = p.cu[k.n];
  k.len = min(64, p.cu[k.n + 1] - lo - k.i * 64);
  k.token = lo + k.i * 64;
  return k;
}

// The sequence that the i-th blocks of a walk take: a walk is as long as its sequence, and one
// that is begun last ends last.  Only behind delta_good().
__device__ __forceinline__ int delta_turn(const DeltaBwdParams &p, int i) {
  return p.cu == nullptr ? i : p.order[i];
}

// The chunks of sequence n: the first one, and how many; 0 with bad offsets.
__device__ __forceinline__ int delta_chunks(const DeltaBwdParams &p, int n, int64_t *first) {
  if (p.cu == nullptr) {
    *first = (int64_t)n * p.per_seq;
    return p.per_seq;
  }
  *first = p.first[n];
  return p.first[n + 1] - p.first[n];
}

// A token's log-gate for the running sums: what lies below e^-104 is zero in float32, and
// sums that pass through lesser values (or through -infinity) would lose the gates behind.
// The sums are formed in 64 bits and kept as two floats, G and what its rounding left: with
// many gates that forget in a chunk they reach thousands, where a float's half step is some
// 1e-4 of e^(G_i - G_j) between tokens that hardly forget.
__device__ __forceinline__ float delta_gate(float g) { return g < -104.f ? -104.f : g; }

// G_i - G_j of sums with their rests.
__device__ __forceinline__ float delta_gap(float Gi, float rest_i, float Gj, float rest_j) {
  return (Gi - Gj) + (rest_i - rest_j);
}
__device__ __forceinline__ float delta_gap(float2 Gi, float2 Gj) {
  return delta_gap(Gi.x, Gi.y, Gj.x, Gj.y);
}

// Of x at a lane's tokens l and l + 32 the sums over the tokens before them; one warp.
__device__ __forceinline__ void delta_before(float (&x)[2]) {
  const int lane = threadIdx.x & 31;
#pragma unroll
  for (int e = 0; e < 2; ++e) {
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const float y = __shfl_up_sync(~0u, x[e], o);
      if (lane >= o) x[e] += y;
    }
  }
  const float half = __shfl_sync(~0u, x[0], 31);
  const float a = __shfl_up_sync(~0u, x[0], 1), b = __shfl_up_sync(~0u, x[1], 1);
  x[0] = lane > 0 ? a : 0.f;
  x[1] = lane > 0 ? half + b : half;
}

// Whether the offsets were good (the table kernel marks bad ones).
__device__ __forceinline__ bool delta_good(const DeltaBwdParams &p) {
  return p.cu == nullptr || p.first[p.N] >= 0;
}
#endif

// Whether the tensor cores take the call, the bytes of a chunk and head, and the launches.
bool delta_bwd_tc_supported(const DeltaBwdParams &p, bool bf16);
int64_t delta_bwd_tc_block(const DeltaBwdParams &p);
int64_t delta_bwd_tc_scratch(const DeltaBwdParams &p);
cudaError_t launch_delta_bwd_tc(const DeltaBwdParams &p, cudaStream_t stream);
int64_t delta_bwd_simt_block(const DeltaBwdParams &p);
cudaError_t launch_delta_bwd_simt(const DeltaBwdParams &p, bool bf16, cudaStream_t stream);

}  // namespace gdn
