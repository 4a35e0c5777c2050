// Norm over groups of channels, shared by its forward and its gradient: how teams of
// threads share the rows, and a team's sums.
//
// A team of threads (a power of two, of one warp or several) holds one token's group in
// registers: PP pieces of VEC channels a thread, `team` pieces apart, so that a warp's loads
// are contiguous.  A team keeps its group and walks tokens, so that its weights stay in L1 and,
// in the gradient, its sums over tokens in registers.  The next tokens' rows are on their way
// while one is computed, and each tensor's place moves on by one addition.
//
// The floor is the rows' bytes, but the instructions come close to it (issue slots 70% full):
// hence arithmetic on two values an instruction, weights in the rows' own type, and kernels of
// their own for groups that threads and pieces divide evenly, without checks of their ends and
// with the team's size known.  bf16: 2 x 4096 tokens of 16 heads of 128 with a gate take 20 us
// (5.0 TB/s of 6.8), 32068 tokens of 8 groups of 512 90 us (5.9 TB/s; 119 in the kernel for
// any group); the gradient of the first 33 us (5.0 TB/s), with 16 warps an SM, as a token's
// values take some 115 registers.  With one
// token ahead, scalar arithmetic and places worked out for every token they took 28.7, 139.6
// and 59.5 us.
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
  int flat;                   // tokens of all batch rows lie one stride apart
  float eps;
  // teams: `team` threads each; `rows` tokens and `span` groups a block, blocks_per_row
  // blocks side by side over the groups; `step` tokens at once
  int team, rows, span, blocks_per_row, step;
};

// A team's place: its group, its first token, and whether it has any.  With TEAM (threads, else
// 0) all comes out even: the teams fill their blocks and the pieces their groups, so that only
// tokens end, and those of all batch rows lie one stride apart.
template <int TEAM>
struct NormTeam {
  int lane, g, t, index;
  bool live;
  static __device__ __forceinline__ int team(const NormParams &p) { return TEAM ? TEAM : p.team; }
  __device__ __forceinline__ explicit NormTeam(const NormParams &p) {
    lane = threadIdx.x & (team(p) - 1);
    index = threadIdx.x / team(p);
    const int row = index / p.span;
    g = blockIdx.x % p.blocks_per_row * p.span + index % p.span;
    t = blockIdx.x / p.blocks_per_row * p.rows + row;
    live = TEAM || (row < p.rows && g < p.G);
  }
  __device__ __forceinline__ bool has(const NormParams &p, int token) const {
    return live && token < p.tokens;
  }
  // whether this thread's piece `from` channels behind its first is one of the group's
  __device__ __forceinline__ bool in(const NormParams &p, int from, int vec) const {
    return TEAM || lane * vec + from < p.W;
  }
};

constexpr int NORM_WARPS = 32;

// Most threads of a block whose threads hold `elements` channels (8192 a group: 16 of them
// want the registers of half the threads).
constexpr int norm_threads(int elements) { return elements > 8 ? 512 : 1024; }
// Threads of an ordinary block; tokens whose rows are on their way and blocks an SM, by the
// words that a thread's part of a row takes (some 48 KB of an SM's are on their way).  Above 8
// channels a thread, us at 52 million values, weights of one group, the choice / the other one:
//   forward, two blocks / three: bf16 with a gate, 512 channels 50 / 56, 1024 68 / 89, 4096 68 / 92;
//     float32, 512 95 / 103, 1024 with a gate 99 / 104, without 81 / 69, 384 141 / 132, 125 / 97;
//     one token ahead / two: float32, 1024 99 / 101
//   backward, one block / two: bf16 with a gate, 512 90 / 100, 1024 174 / 212, float32, 1024
//     190 / 291; without a gate two would be faster: bf16, 512 81 / 62, 1024 152 / 119, float32,
//     1024 163 / 138 (512, whose ring takes an SM, 117 / 127); one token ahead / two: float32,
//     1024 190 / 243, bf16 174 / 176
constexpr int NORM_THREADS = 256;
constexpr int norm_words(int elt, int vec, int pieces) {
  return pieces * (vec * elt >= 4 ? vec * elt / 4 : 1);
}
constexpr int norm_fwd_ahead(int words, bool z) { return words > 8 ? 1 : words > 4 || z ? 2 : 3; }
constexpr int norm_fwd_per_sm(int elements, int words, bool z) {
  return words > 8 || (elements > 8 && z) ? 2 : words > 4 || z ? 3 : elements > 2 ? 4 : 6;
}
// (of the gradient's kernels for any group; the even ones have a ring)
constexpr int norm_bwd_ahead(int words) { return words > 4 ? 1 : 2; }
constexpr int norm_bwd_per_sm(int elements) { return elements > 8 ? 1 : elements > 2 ? 2 : 4; }
// A block's threads: NORM_THREADS, or what the widest groups want.
constexpr int norm_block(int elements, bool wide) {
  return wide ? norm_threads(elements) : NORM_THREADS;
}
// Most pieces a thread takes.
constexpr int norm_pieces(int vec) { return vec == 8 ? 2 : vec == 4 ? 4 : 8; }

// v summed over the team, for all its threads; the whole block takes part.  `buf` holds two
// sets of a block's warps' sums, taken in turn, so that one barrier a call is enough.
template <int N>
__device__ __forceinline__ void team_sum(float (&v)[N], int team, float (*buf)[NORM_WARPS][2],
                                         int &turn) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1)
    if (team > o)
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

// Element-wise operations on VEC values, two an instruction where there are two.
template <int VEC>
__device__ __forceinline__ void vmul(float *out, const float *a, const float *b) {
  if constexpr (VEC == 1)
    out[0] = a[0] * b[0];
  else
    mul_row<VEC>(out, a, b);
}
template <int VEC>
__device__ __forceinline__ void vmul(float *out, const float *a, float f) {
  const float b[2] = {f, f};
#pragma unroll
  for (int e = 0; e < VEC; e += 2) vmul<VEC == 1 ? 1 : 2>(out + e, a + e, b);
}
template <int VEC>
__device__ __forceinline__ void vadd(float *out, const float *a, const float *b) {
  if constexpr (VEC == 1)
    out[0] = a[0] + b[0];
  else
    add_row<VEC>(out, a, b);
}
template <int VEC>
__device__ __forceinline__ void vsub(float *out, const float *a, float f) {
  const float b[2] = {f, f};
#pragma unroll
  for (int e = 0; e < VEC; e += 2) {
    if constexpr (VEC == 1)
      out[0] = a[0] - f;
    else
      sub_row<2>(out + e, a + e, b);
  }
}
// out = a b + c, and with one factor for all
template <int VEC>
__device__ __forceinline__ void vfma(float *out, const float *a, const float *b, const float *c) {
  if constexpr (VEC == 1)
    out[0] = fmaf(a[0], b[0], c[0]);
  else
    fma_rows<VEC>(out, a, b, c);
}
template <int VEC>
__device__ __forceinline__ void vfma(float *out, const float *a, float f, const float *c) {
  const float b[2] = {f, f};
#pragma unroll
  for (int e = 0; e < VEC; e += 2) vfma<VEC == 1 ? 1 : 2>(out + e, a + e, b, c + e);
}
// Two partial sums of products, and of values.
template <int VEC>
__device__ __forceinline__ void vdot(float (&sum)[2], const float *a, const float *b) {
#pragma unroll
  for (int e = 0; e < VEC; e += 2) vfma<VEC == 1 ? 1 : 2>(sum, a + e, b + e, sum);
}
template <int VEC>
__device__ __forceinline__ void vsum(float (&sum)[2], const float *a) {
#pragma unroll
  for (int e = 0; e < VEC; e += 2) vadd<VEC == 1 ? 1 : 2>(sum, sum, a + e);
}

// act(z) (out may be z), and its derivative where wanted: s (1 + z (1 - s)) or s (1 - s) with
// s = 1 / (1 + e^-z).
template <int VEC, bool SLOPE>
__device__ __forceinline__ void norm_act(int act, const float *z, float *out, float *slope) {
  if (act == GDN_ACT_NONE) {
#pragma unroll
    for (int e = 0; e < VEC; ++e) {
      out[e] = z[e];
      if (SLOPE) slope[e] = 1.f;
    }
    return;
  }
  float s[VEC];
  if constexpr (VEC == 1)
    s[0] = __fdividef(1.f, 1.f + __expf(-z[0]));
  else
    sigmoid_row<VEC>(s, z);
  [[maybe_unused]] float rest[VEC];
  if constexpr (SLOPE) {  // 1 - s
    float less[VEC], one[VEC];
#pragma unroll
    for (int e = 0; e < VEC; ++e) less[e] = -1.f, one[e] = 1.f;
    vfma<VEC>(rest, s, less, one);
  }
  if (act == GDN_ACT_SILU) {
    vmul<VEC>(out, z, s);
    if constexpr (SLOPE) vfma<VEC>(slope, out, rest, s);
  } else {
    if constexpr (SLOPE) vmul<VEC>(slope, s, rest);
#pragma unroll
    for (int e = 0; e < VEC; ++e) out[e] = s[e];
  }
}

// A team's weights or biases: a piece of them (zero past the group) lies as wide as the rows'.
// KEEP: those of the rows' own type stay in registers; others are read for every token, from L1.
template <typename T, int VEC, int PP, bool KEEP>
struct NormWeights {
  const unsigned char *at;  // NULL: none
  int step;                 // bytes from piece to piece
  Row<T, VEC> kept[KEEP ? PP : 1];
  template <int TEAM>
  __device__ __forceinline__ NormWeights(const NormParams &p, const NormTeam<TEAM> &m, const void *from) {
    const int size = p.w_f32 ? 4 : (int)sizeof(T);
    at = static_cast<const unsigned char *>(from);
    if (at != nullptr) at += ((p.shared ? 0 : (int64_t)m.g * p.W) + m.lane * VEC) * size;
    step = VEC * m.team(p) * size;
    if constexpr (KEEP) {
#pragma unroll
      for (int j = 0; j < PP; ++j) {
        kept[j].zero();
        if (at != nullptr && !p.w_f32 && m.live && m.in(p, j * VEC * m.team(p), VEC))
          kept[j].load(reinterpret_cast<const T *>(at + j * step));
      }
    }
  }
  template <int TEAM>
  __device__ __forceinline__ void get(const NormParams &p, const NormTeam<TEAM> &m, int piece, float *w) const {
    if (KEEP && !p.w_f32) return kept[KEEP ? piece : 0].widen(w);
    if (!m.live || !m.in(p, piece * VEC * m.team(p), VEC)) {
#pragma unroll
      for (int e = 0; e < VEC; ++e) w[e] = 0.f;
      return;
    }
    const unsigned char *here = at + piece * step;
    if (p.w_f32) {
      constexpr int N = VEC >= 4 ? 4 : VEC;
#pragma unroll
      for (int e = 0; e < VEC; e += N) {
        Row<float, N> r;
        r.load(reinterpret_cast<const float *>(here) + e);
        r.widen(w + e);
      }
    } else {
      Row<T, VEC> r;
      r.load(reinterpret_cast<const T *>(here));
      r.widen(w);
    }
  }
};

// A team's way through one tensor: where the next token's pieces of it are.  (A place is
// worked out once where tokens lie one stride apart, as with TEAM, then moved on.)
template <typename T, int TEAM>
struct NormCursor {
  T *at;
  int64_t stride, batch, move;
  __device__ __forceinline__ NormCursor(const NormParams &p, const NormTeam<TEAM> &m,
                                        const void *base, int64_t stride_, int64_t batch_, int vec)
      : stride(stride_), batch(batch_), move(p.step * stride_) {
    at = static_cast<T *>(const_cast<void *>(base)) + (int64_t)m.g * p.W + m.lane * vec;
    if (TEAM || p.flat) at += m.t * stride;
  }
  // token t's place (of tokens taken in turn)
  __device__ __forceinline__ T *next(const NormParams &p, int t) {
    if (TEAM || p.flat) {
      T *here = at;
      at += move;
      return here;
    }
    const int b = t / p.T;
    return at + b * batch + (t - b * p.T) * stride;
  }
};

// A token's pieces of one tensor, as they lie in memory; of token t where it is `there`.
template <typename T, int VEC, int PP>
struct NormRow {
  Row<T, VEC> r[PP];
  template <int TEAM>
  __device__ __forceinline__ void load(const NormParams &p, const NormTeam<TEAM> &m,
                                       NormCursor<T, TEAM> &c, int t, bool there) {
    const T *at = c.next(p, t);
#pragma unroll
    for (int j = 0; j < PP; ++j)
      if (there && m.in(p, j * VEC * m.team(p), VEC)) r[j].load(at + j * VEC * m.team(p));
  }
  template <int TEAM>
  __device__ __forceinline__ void store(const NormParams &p, const NormTeam<TEAM> &m,
                                        NormCursor<T, TEAM> &c, int t, bool there) const {
    T *at = c.next(p, t);
#pragma unroll
    for (int j = 0; j < PP; ++j)
      if (there && m.in(p, j * VEC * m.team(p), VEC)) r[j].store(at + j * VEC * m.team(p));
  }
  __device__ __forceinline__ void zero() {
#pragma unroll
    for (int j = 0; j < PP; ++j) r[j].zero();
  }
};

// Takes u's mean off (where wanted) and returns 1 / root.  Pieces past the group hold zero and
// stay so.
template <int VEC, int PP, int TEAM>
__device__ __forceinline__ float norm_root(const NormParams &p, const NormTeam<TEAM> &m,
                                           float (&u)[PP][VEC], float (*buf)[NORM_WARPS][2],
                                           int &turn) {
  const float inv = 1.f / (float)p.W;
  float v[1];
  if (p.center) {
    float s[2] = {0.f, 0.f};
#pragma unroll
    for (int j = 0; j < PP; ++j) vsum<VEC>(s, u[j]);
    v[0] = s[0] + s[1];
    team_sum(v, m.team(p), buf, turn);
    const float mean = v[0] * inv;
#pragma unroll
    for (int j = 0; j < PP; ++j)
      if (m.in(p, j * VEC * m.team(p), VEC)) vsub<VEC>(u[j], u[j], mean);
  }
  float s[2] = {0.f, 0.f};
#pragma unroll
  for (int j = 0; j < PP; ++j) vdot<VEC>(s, u[j], u[j]);
  v[0] = s[0] + s[1];
  team_sum(v, m.team(p), buf, turn);
  return rsqrtf(fmaf(v[0], inv, p.eps));
}

// How a call is shared out: channels a piece, pieces a thread, threads a block, blocks, and a
// team's threads where all comes out even and a kernel is made for as many (else 0).
struct NormPlan {
  int vec, pieces, threads, blocks, team;
};
cudaError_t launch_norm_fwd(const NormParams &p, bool bf16, const NormPlan &plan, cudaStream_t stream);
cudaError_t launch_norm_bwd(const NormParams &p, bool bf16, const NormPlan &plan, cudaStream_t stream);
// dw and db (or NULL) [columns] from part [rows][2][columns].
cudaError_t launch_norm_sums(const float *part, int rows, int columns, float *dw, float *db,
                             cudaStream_t stream);

// Where z stands.
enum NormGate { NO_GATE, GATE_AFTER, GATE_BEFORE };

// Calls f with the element type, VEC, PP, the gate and TEAM as compile-time values.  TEAM is for
// pieces of 16 bytes, teams of 8 to 32 threads (groups of 64 channels and more in bfloat16),
// of 32 where a thread takes several pieces.
template <typename F>
cudaError_t norm_forms(bool bf16, const NormPlan &plan, const NormParams &p, F &&f) {
  auto gate = [&](auto t, auto v, auto n, auto team) {
    if (p.z == nullptr) return f(t, v, n, std::integral_constant<NormGate, NO_GATE>(), team);
    if (p.gate_first) return f(t, v, n, std::integral_constant<NormGate, GATE_BEFORE>(), team);
    return f(t, v, n, std::integral_constant<NormGate, GATE_AFTER>(), team);
  };
  const std::integral_constant<int, 0> any;
  const int pieces = plan.pieces;
  auto one = [&](auto t, auto v) {
    const std::integral_constant<int, 1> n;
    if (plan.team == 8) return gate(t, v, n, std::integral_constant<int, 8>());
    if (plan.team == 16) return gate(t, v, n, std::integral_constant<int, 16>());
    if (plan.team == 32) return gate(t, v, n, std::integral_constant<int, 32>());
    return gate(t, v, n, any);
  };
  auto several = [&](auto t, auto v, auto n) {
    if (plan.team == 32) return gate(t, v, n, std::integral_constant<int, 32>());
    return gate(t, v, n, any);
  };
  auto few = [&](auto t, auto v) {  // PP of 1, 2 (and 4 for four channels a piece)
    if (pieces == 1) return one(t, v);
    if (decltype(v)::value == 8 || pieces == 2)
      return several(t, v, std::integral_constant<int, 2>());
    return several(t, v, std::integral_constant<int, decltype(v)::value == 8 ? 2 : 4>());
  };
  auto many = [&](auto t, auto v) {
    if (pieces == 1) return gate(t, v, std::integral_constant<int, 1>(), any);
    if (pieces == 2) return gate(t, v, std::integral_constant<int, 2>(), any);
    if (pieces == 4) return gate(t, v, std::integral_constant<int, 4>(), any);
    if (pieces == 6) return gate(t, v, std::integral_constant<int, 6>(), any);
    return gate(t, v, std::integral_constant<int, 8>(), any);
  };
  if (bf16) {
    if (plan.vec == 8) return few(__nv_bfloat16(), std::integral_constant<int, 8>());
    if (plan.vec == 2) return many(__nv_bfloat16(), std::integral_constant<int, 2>());
    return many(__nv_bfloat16(), std::integral_constant<int, 1>());
  }
  if (plan.vec == 4) return few(0.f, std::integral_constant<int, 4>());
  return many(0.f, std::integral_constant<int, 1>());
}

}  // namespace gdn
