// Norm over groups of channels, shared by its forward and its gradient: how teams of
// threads share the rows, and a team's sums.
//
// A team of threads (a power of two, of one warp or several) holds one token's group in
// registers: PP pieces of VEC channels a thread, `team` pieces apart, so that a warp's loads
// are contiguous.  A team keeps its group and walks tokens, so that its weights are loaded
// once and, in the gradient, its sums over tokens stay in registers.  The next token's rows
// are on their way while one is computed: the operator is bound by memory.
#pragma once

#include <type_traits>

#include "rows.cuh"

namespace gdn {

struct NormParams {
  const void *dy, *x, *z, *weight, *bias;
  void *y, *dz;               // y: dx of the gradient
  float *part;                // [rows][2][columns] partial sums of dweight and dbias, or NULL
  int *err;
  int64_t gs, gb, xs, xb, zs, zb, ys, yb, ds, db;
  int tokens, T, G, W, D;     // all tokens, tokens of a batch row
  int shared, w_f32, center, gate_first, act;
  float eps;
  // teams: `team` threads each; `rows` tokens and `span` groups a block, blocks_per_row
  // blocks side by side over the groups; `step` tokens at once
  int team, rows, span, blocks_per_row, step;
};

// A team's place: its group, its first token, and whether it has any.
struct NormTeam {
  int lane, g, t, index;
  bool live;
  __device__ __forceinline__ explicit NormTeam(const NormParams &p) {
    lane = threadIdx.x & (p.team - 1);
    index = threadIdx.x / p.team;
    const int row = index / p.span;
    g = blockIdx.x % p.blocks_per_row * p.span + index % p.span;
    t = blockIdx.x / p.blocks_per_row * p.rows + row;
    live = row < p.rows && g < p.G;
  }
};

constexpr int NORM_WARPS = 32;

// Most threads of a block whose threads hold `elements` channels (8192 a group: 16 of them
// want the registers of half the threads).
constexpr int norm_threads(int elements) { return elements > 8 ? 512 : 1024; }
// Threads of an ordinary block, and the blocks that an SM holds of them.
constexpr int NORM_FWD_THREADS = 256, NORM_BWD_THREADS = 256;
constexpr int norm_fwd_per_sm(int elements) { return elements > 8 ? 2 : elements > 2 ? 4 : 8; }
constexpr int norm_bwd_per_sm(int elements) { return elements > 8 ? 1 : elements > 2 ? 2 : 4; }
// Most pieces a thread takes.
constexpr int norm_pieces(int vec) { return vec == 8 ? 2 : vec == 4 ? 4 : 8; }

// v summed over the team, for all its threads; the whole block takes part.  `buf` holds two
// sets of a block's warps' sums, taken in turn, so that one barrier a call is enough.
template <int N>
__device__ __forceinline__ void team_sum(float (&v)[N], int team, float (*buf)[NORM_WARPS][2],
                                         int &turn) {
  for (int o = min(team, 32) >> 1; o > 0; o >>= 1)
#pragma unroll
    for (int i = 0; i < N; ++i) v[i] += __shfl_xor_sync(~0u, v[i], o);
  if (team <= 32) return;
  const int warp = threadIdx.x >> 5, each = team >> 5, first = warp / each * each;
  if ((threadIdx.x & 31) == 0)
#pragma unroll
    for (int i = 0; i < N; ++i) buf[turn][warp][i] = v[i];
  __syncthreads();
#pragma unroll
  for (int i = 0; i < N; ++i) v[i] = 0.f;
  for (int k = 0; k < each; ++k)
#pragma unroll
    for (int i = 0; i < N; ++i) v[i] += buf[turn][first + k][i];
  turn ^= 1;
}

// 1 / (1 + e^-z) of VEC values (two an instruction where there are two)
template <int VEC>
__device__ __forceinline__ void norm_sigmoid(float *out, const float *z) {
  if constexpr (VEC == 1)
    out[0] = __fdividef(1.f, 1.f + __expf(-z[0]));
  else
    sigmoid_row<VEC>(out, z);
}

// act(z), and its derivative where wanted
template <int VEC>
__device__ __forceinline__ void norm_act(int act, const float *z, float *out, float *slope) {
  float s[VEC];
  if (act == GDN_ACT_NONE) {
#pragma unroll
    for (int e = 0; e < VEC; ++e) {
      out[e] = z[e];
      if (slope) slope[e] = 1.f;
    }
    return;
  }
  norm_sigmoid<VEC>(s, z);
#pragma unroll
  for (int e = 0; e < VEC; ++e) {
    const float v = z[e];  // (out may be z)
    out[e] = act == GDN_ACT_SILU ? v * s[e] : s[e];
    if (slope) slope[e] = s[e] * fmaf(act == GDN_ACT_SILU ? v : 1.f, 1.f - s[e],
                                      act == GDN_ACT_SILU ? 1.f : 0.f);
  }
}

// Weights or biases of a team's channels (`none` where there are none).
template <typename T, int VEC, int PP>
__device__ __forceinline__ void norm_weights(const NormParams &p, const NormTeam &m,
                                             const void *from, float none, float (&w)[PP][VEC]) {
  const int base = p.shared ? 0 : m.g * p.W;
#pragma unroll
  for (int j = 0; j < PP; ++j) {
    const int c = (m.lane + j * p.team) * VEC;
#pragma unroll
    for (int e = 0; e < VEC; ++e) w[j][e] = none;
    if (from == nullptr || !m.live || c >= p.W) continue;
#pragma unroll
    for (int e = 0; e < VEC; ++e)
      w[j][e] = p.w_f32 ? static_cast<const float *>(from)[base + c + e]
                        : to_f32(static_cast<const T *>(from)[base + c + e]);
  }
}

// A token's pieces of one tensor, as they lie in memory.
template <typename T, int VEC, int PP>
struct NormRow {
  Row<T, VEC> r[PP];
  __device__ __forceinline__ void load(const NormParams &p, const NormTeam &m, const void *base,
                                       int64_t stride, int64_t batch, int t) {
    if (!m.live || t >= p.tokens) return;
    const int b = t / p.T;
    const T *at = static_cast<const T *>(base) + b * batch + (t - b * p.T) * stride +
                  (int64_t)m.g * p.W;
#pragma unroll
    for (int j = 0; j < PP; ++j) {
      const int c = (m.lane + j * p.team) * VEC;
      if (c < p.W) r[j].load(at + c);
    }
  }
  __device__ __forceinline__ void store(const NormParams &p, const NormTeam &m, void *base,
                                        int64_t stride, int64_t batch, int t) const {
    if (!m.live || t >= p.tokens) return;
    const int b = t / p.T;
    T *at = static_cast<T *>(base) + b * batch + (t - b * p.T) * stride + (int64_t)m.g * p.W;
#pragma unroll
    for (int j = 0; j < PP; ++j) {
      const int c = (m.lane + j * p.team) * VEC;
      if (c < p.W) r[j].store(at + c);
    }
  }
  __device__ __forceinline__ void zero() {
#pragma unroll
    for (int j = 0; j < PP; ++j) r[j].zero();
  }
};

// u to its normal form in place; returns 1 / root.  Pieces past the group hold zero and
// stay so.
template <int VEC, int PP>
__device__ __forceinline__ float normalise(const NormParams &p, const NormTeam &m,
                                           float (&u)[PP][VEC], float (*buf)[NORM_WARPS][2],
                                           int &turn) {
  const float inv = 1.f / (float)p.W;
  float s[1] = {0.f};
  if (p.center) {
#pragma unroll
    for (int j = 0; j < PP; ++j)
#pragma unroll
      for (int e = 0; e < VEC; ++e) s[0] += u[j][e];
    team_sum(s, p.team, buf, turn);
    const float mean = s[0] * inv;
#pragma unroll
    for (int j = 0; j < PP; ++j)
      if ((m.lane + j * p.team) * VEC < p.W)
#pragma unroll
        for (int e = 0; e < VEC; ++e) u[j][e] -= mean;
    s[0] = 0.f;
  }
#pragma unroll
  for (int j = 0; j < PP; ++j)
#pragma unroll
    for (int e = 0; e < VEC; ++e) s[0] = fmaf(u[j][e], u[j][e], s[0]);
  team_sum(s, p.team, buf, turn);
  const float r = 1.f / sqrtf(fmaf(s[0], inv, p.eps));
#pragma unroll
  for (int j = 0; j < PP; ++j)
    if ((m.lane + j * p.team) * VEC < p.W)
#pragma unroll
      for (int e = 0; e < VEC; ++e) u[j][e] *= r;
  return r;
}

cudaError_t launch_norm_fwd(const NormParams &p, bool bf16, int vec, int pieces, int threads,
                            int blocks, cudaStream_t stream);
cudaError_t launch_norm_bwd(const NormParams &p, bool bf16, int vec, int pieces, int threads,
                            int blocks, cudaStream_t stream);
// dw and db (or NULL) [columns] from part [rows][2][columns].
cudaError_t launch_norm_sums(const float *part, int rows, int columns, float *dw, float *db,
                             cudaStream_t stream);

// Calls f with the element type, VEC, PP and whether there is a z as compile-time values.
template <typename F>
cudaError_t norm_forms(bool bf16, int vec, int pieces, bool z, F &&f) {
  auto gate = [&](auto t, auto v, auto n) {
    return z ? f(t, v, n, std::true_type()) : f(t, v, n, std::false_type());
  };
  auto few = [&](auto t, auto v) {  // PP of 1, 2 (and 4 for four channels a piece)
    if (pieces == 1) return gate(t, v, std::integral_constant<int, 1>());
    if (decltype(v)::value == 8 || pieces == 2) return gate(t, v, std::integral_constant<int, 2>());
    return gate(t, v, std::integral_constant<int, decltype(v)::value == 8 ? 2 : 4>());
  };
  auto many = [&](auto t, auto v) {
    if (pieces == 1) return gate(t, v, std::integral_constant<int, 1>());
    if (pieces == 2) return gate(t, v, std::integral_constant<int, 2>());
    if (pieces == 4) return gate(t, v, std::integral_constant<int, 4>());
    if (pieces == 6) return gate(t, v, std::integral_constant<int, 6>());
    return gate(t, v, std::integral_constant<int, 8>());
  };
  if (bf16) {
    if (vec == 8) return few(__nv_bfloat16(), std::integral_constant<int, 8>());
    if (vec == 2) return many(__nv_bfloat16(), std::integral_constant<int, 2>());
    return many(__nv_bfloat16(), std::integral_constant<int, 1>());
  }
  if (vec == 4) return few(0.f, std::integral_constant<int, 4>());
  return many(0.f, std::integral_constant<int, 1>());
}

}  // namespace gdn
