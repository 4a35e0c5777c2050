// Norm over groups of channels of every token, with its activation or gate: the forward
// kernel, the argument checks and the entry points of both directions.  The gradient's
// kernels are in group_norm_bwd.cu.
#include <math.h>

#include <algorithm>
#include <initializer_list>
#include <type_traits>

#include "abi_check.h"
#include "group_norm.cuh"

namespace gdn {
namespace {

template <typename T, int VEC, int PP, bool Z, int TEAM, bool WIDE>
__global__ void __launch_bounds__(
    norm_block(PP * VEC, WIDE),
    WIDE ? 1 : norm_fwd_per_sm(PP * VEC, norm_words(sizeof(T), VEC, PP), Z))
norm_fwd_kernel(NormParams p) {
  constexpr int AHEAD = WIDE ? 1 : norm_fwd_ahead(norm_words(sizeof(T), VEC, PP), Z);
  __shared__ float buf[2][NORM_WARPS][2];
  const NormTeam<TEAM> m(p);
  if (!bounds_ok(p.team * p.rows * p.span <= (int)blockDim.x, p.err)) return;
  int turn = 0;
  NormCursor<T, TEAM> xc(p, m, p.x, p.xs, p.xb, VEC), zc(p, m, p.z, p.zs, p.zb, VEC);
  NormCursor<T, TEAM> yc(p, m, p.y, p.ys, p.yb, VEC);
  const NormWeights<T, VEC, PP, false> weight(p, m, p.weight), bias(p, m, p.bias);
  NormRow<T, VEC, PP> x[AHEAD], z[Z ? AHEAD : 1];
#pragma unroll
  for (int i = 0; i < AHEAD; ++i) {
    x[i].zero();
    const int t = m.t + i * p.step;
    x[i].load(p, m, xc, t, m.has(p, t));
    if constexpr (Z) {
      z[i].zero();
      z[i].load(p, m, zc, t, m.has(p, t));
    }
  }
  // every team of a block takes as many turns: the sums are the block's
  const int first = blockIdx.x / p.blocks_per_row * p.rows;
  for (int t0 = first, t = m.t; t0 < p.tokens;) {
#pragma unroll
    for (int i = 0; i < AHEAD; ++i, t0 += p.step, t += p.step) {
      if (t0 >= p.tokens) break;
      float u[PP][VEC], gate[Z ? PP : 1][VEC];
#pragma unroll
      for (int j = 0; j < PP; ++j) {
        x[i].r[j].widen(u[j]);
        if constexpr (Z) {
          z[i].r[j].widen(gate[j]);
          norm_act<VEC, false>(p.act, gate[j], gate[j], nullptr);
          if (p.gate_first) vmul<VEC>(u[j], u[j], gate[j]);
        }
      }
      const int later = t + AHEAD * p.step;
      const bool more = m.has(p, later);
      x[i].load(p, m, xc, later, more);
      if constexpr (Z) z[i].load(p, m, zc, later, more);
      const float r = norm_root<VEC, PP>(p, m, u, buf, turn);
      NormRow<T, VEC, PP> y;
#pragma unroll
      for (int j = 0; j < PP; ++j) {
        vmul<VEC>(u[j], u[j], r);
        if (p.weight != nullptr) {
          float w[VEC];
          weight.get(p, m, j, w);
          vmul<VEC>(u[j], u[j], w);
        }
        if (p.bias != nullptr) {
          float b[VEC];
          bias.get(p, m, j, b);
          vadd<VEC>(u[j], u[j], b);
        }
        if constexpr (Z) {
          if (!p.gate_first) vmul<VEC>(u[j], u[j], gate[j]);
        } else {
          norm_act<VEC, false>(p.act, u[j], u[j], nullptr);
        }
        y.r[j].round(u[j]);
      }
      y.store(p, m, yc, t, m.has(p, t));
    }
  }
}

// ---------------------------------------------------------------- host

// `t` passes the last token by a few steps of less than 2^18, and has to stay within 31 bits.
constexpr int64_t NORM_MAX_TOKENS = MAX_TOKENS - (1 << 20);

NormPlan norm_plan(NormParams &p, bool bf16, int vec, bool bwd) {
  const int all = p.W / vec, most = norm_pieces(vec);
  // as few pieces a thread as keep a group within a warp, where that can be
  int n = 1;
  while (n < most && (all + n - 1) / n > 32) n += n < 4 ? n : 2;
  p.team = 1;
  while (p.team * n < all) p.team *= 2;
  NormPlan plan{vec, n, std::max(NORM_THREADS, p.team), 0, 0};
  const int per_sm = bwd ? norm_bwd_per_sm(vec * n)
                         : norm_fwd_per_sm(vec * n, norm_words(bf16 ? 2 : 4, vec, n), p.z != nullptr);
  const int teams = plan.threads / p.team;
  p.span = std::min(teams, p.G);
  p.blocks_per_row = (p.G + p.span - 1) / p.span;
  p.rows = teams / p.span;
  // blocks that are on the GPU at once, and no more than have tokens
  const int64_t held = std::max<int64_t>(1, (int64_t)sm_count() * per_sm / p.blocks_per_row);
  const int64_t wanted = (p.tokens + p.rows - 1) / p.rows;
  const int64_t down = std::max<int64_t>(1, std::min(held, wanted));
  p.step = (int)down * p.rows;
  plan.blocks = (int)(down * p.blocks_per_row);
  const bool even = p.flat && p.team * n == all && teams == p.rows * p.span && p.G % p.span == 0;
  const bool made = p.team == 32 || (n == 1 && (p.team == 8 || p.team == 16));
  plan.team = even && made && vec * (bf16 ? 2 : 4) == 16 ? p.team : 0;
  return plan;
}

// The widest pieces that divide a group and that every row begins on.
int norm_vec(const NormParams &p, bool bf16, std::initializer_list<const void *> tensors,
             std::initializer_list<int64_t> strides) {
  const int elt = bf16 ? 2 : 4;
  for (int vec = 16 / elt; vec > 1; vec = bf16 && vec == 8 ? 2 : 1) {
    bool ok = p.W % vec == 0;
    for (const void *w : {p.weight, p.bias})  // a piece of them, in loads of 16 bytes at most
      ok = ok && aligned_to(w, std::min(vec * (p.w_f32 ? 4 : elt), 16));
    for (const void *t : tensors) ok = ok && aligned_to(t, vec * elt);
    for (int64_t s : strides) ok = ok && s % vec == 0;
    if (ok) return vec;
  }
  return 1;
}

template <typename Args>
gdn_status_t check_norm(const Args &a) {
  CHECK_DTYPE(a.dtype, "dtype");
  CHECK_DTYPE(a.weight_dtype, "weight_dtype");
  CHECK_THAT(a.weight_dtype == GDN_F32 || a.weight_dtype == a.dtype, GDN_ERR_INVALID_ARG,
             "weight_dtype must be GDN_F32 or dtype");
  CHECK_THAT(a.B >= 1 && a.T >= 0 && a.D >= 1 && a.groups >= 1, GDN_ERR_INVALID_ARG,
             "sizes must be positive (B=%d T=%d D=%d groups=%d)", a.B, a.T, a.D, a.groups);
  CHECK_THAT(a.D % a.groups == 0, GDN_ERR_INVALID_ARG, "D (%d) must be a multiple of groups (%d)",
             a.D, a.groups);
  CHECK_THAT(a.D / a.groups <= 8192, GDN_ERR_UNSUPPORTED, "groups of %d channels exceed 8192",
             a.D / a.groups);
  CHECK_THAT(a.D <= (1 << 28), GDN_ERR_UNSUPPORTED, "D (%d) must be at most %d", a.D, 1 << 28);
  CHECK_THAT((int64_t)a.B * a.T <= NORM_MAX_TOKENS, GDN_ERR_UNSUPPORTED,
             "B * T (%lld) must be at most %lld", (long long)a.B * a.T, (long long)NORM_MAX_TOKENS);
  CHECK_FLAG(a.shared_weight, "shared_weight");
  CHECK_FLAG(a.center, "center");
  CHECK_FLAG(a.gate_first, "gate_first");
  CHECK_THAT(a.activation >= GDN_ACT_NONE && a.activation <= GDN_ACT_SIGMOID, GDN_ERR_INVALID_ARG,
             "activation %d is not a gdn_activation_t", a.activation);
  CHECK_THAT(isfinite(a.eps) && a.eps >= 0.f, GDN_ERR_INVALID_ARG, "eps must be finite and not negative");
  CHECK_THAT(!a.gate_first || a.z != nullptr, GDN_ERR_INVALID_ARG, "gate_first needs z");
  if (a.weight != nullptr) CHECK_TOKENS(a.weight, "weight", a.weight_dtype);
  if (a.bias != nullptr) CHECK_TOKENS(a.bias, "bias", a.weight_dtype);
  if (a.B * (int64_t)a.T > 0) {
    CHECK_TOKENS(a.x, "x", a.dtype);
    if (a.z != nullptr) CHECK_TOKENS(a.z, "z", a.dtype);
    CHECK_THAT(a.x_stride >= a.D && (a.z == nullptr || a.z_stride >= a.D), GDN_ERR_INVALID_ARG,
               "a token stride is less than its row");
  }
  return GDN_OK;
}

// A stride that no second token or batch row uses may be anything.
template <typename Args>
NormParams norm_params(const Args &a) {
  NormParams p{};
  const bool tokens = a.T > 1, many = a.B > 1;
  p.x = a.x; p.z = a.z; p.weight = a.weight; p.bias = a.bias;
  p.xs = tokens ? a.x_stride : a.D; p.xb = many ? a.x_batch_stride : 0;
  p.zs = tokens && a.z ? a.z_stride : a.D; p.zb = many && a.z ? a.z_batch_stride : 0;
  p.tokens = a.B * a.T; p.T = a.T;
  p.G = a.groups; p.W = a.D / a.groups; p.D = a.D;
  p.shared = a.shared_weight; p.w_f32 = a.weight_dtype == GDN_F32;
  p.flat = a.B == 1;
  p.center = a.center; p.gate_first = a.gate_first; p.act = a.activation; p.eps = a.eps;
  return p;
}

// Whether a tensor's batch rows follow one another.
bool evenly(const NormParams &p, int64_t stride, int64_t batch) { return batch == p.T * stride; }

gdn_status_t check_bwd(const group_norm_bwd_args &a) {
  gdn_status_t st = check_norm(a);
  if (st != GDN_OK) return st;
  if (a.B * (int64_t)a.T > 0) {
    CHECK_TOKENS(a.dy, "dy", a.dtype);
    CHECK_TOKENS(a.dx, "dx", a.dtype);
    CHECK_THAT(a.dy_stride >= a.D && a.dx_stride >= a.D && (a.z == nullptr || a.dz_stride >= a.D),
               GDN_ERR_INVALID_ARG, "a token stride is less than its row");
    CHECK_THAT((a.z != nullptr) == (a.dz != nullptr), GDN_ERR_INVALID_ARG,
               "dz must be given exactly when z is");
    if (a.dz != nullptr) CHECK_TOKENS(a.dz, "dz", a.dtype);
  }
  CHECK_THAT(a.dweight == nullptr || a.weight != nullptr, GDN_ERR_INVALID_ARG,
             "dweight needs a weight");
  CHECK_THAT(a.dbias == nullptr || a.bias != nullptr, GDN_ERR_INVALID_ARG, "dbias needs a bias");
  CHECK_OPT_PTR(a.dweight, "dweight");
  CHECK_OPT_PTR(a.dbias, "dbias");
  return GDN_OK;
}

NormPlan bwd_plan(const group_norm_bwd_args &a, NormParams &p) {
  const bool tokens = a.T > 1, many = a.B > 1, bf16 = a.dtype == GDN_BF16;
  p.dy = a.dy; p.y = a.dx; p.dz = a.dz;
  p.gs = tokens ? a.dy_stride : a.D; p.gb = many ? a.dy_batch_stride : 0;
  p.ys = tokens ? a.dx_stride : a.D; p.yb = many ? a.dx_batch_stride : 0;
  p.ds = tokens && a.z ? a.dz_stride : a.D; p.db = many && a.z ? a.dz_batch_stride : 0;
  const bool z = p.z != nullptr;
  p.flat = p.flat || (evenly(p, p.gs, p.gb) && evenly(p, p.xs, p.xb) && evenly(p, p.ys, p.yb) &&
                      (!z || (evenly(p, p.zs, p.zb) && evenly(p, p.ds, p.db))));
  const int vec = norm_vec(p, bf16, {p.dy, p.x, p.z, p.y, p.dz},
                           {p.gs, p.gb, p.xs, p.xb, p.zs, p.zb, p.ys, p.yb, p.ds, p.db});
  return norm_plan(p, bf16, vec, true);
}

int part_columns(const NormParams &p) { return p.shared ? p.W : p.D; }

int part_rows(const NormParams &p, const NormPlan &plan) {
  return p.shared ? plan.blocks : plan.blocks / p.blocks_per_row;
}

size_t bwd_workspace(const group_norm_bwd_args &a, const NormParams &p, const NormPlan &plan) {
  if (p.tokens == 0 || (a.dweight == nullptr && a.dbias == nullptr)) return 0;
  return (size_t)part_rows(p, plan) * 2 * part_columns(p) * sizeof(float);
}

}  // namespace

cudaError_t launch_norm_fwd(const NormParams &p, bool bf16, const NormPlan &plan, cudaStream_t stream) {
  return norm_forms(bf16, plan, p, [&](auto t, auto v, auto n, auto gate, auto team) {
    using T = decltype(t);
    constexpr int VEC = decltype(v)::value, PP = decltype(n)::value;
    constexpr bool Z = decltype(gate)::value != NO_GATE;
    constexpr int TEAM = decltype(team)::value;
    if (plan.threads <= NORM_THREADS) {
      norm_fwd_kernel<T, VEC, PP, Z, TEAM, false><<<plan.blocks, plan.threads, 0, stream>>>(p);
    } else {  // only with the most pieces a thread
      if constexpr (PP == norm_pieces(VEC))
        norm_fwd_kernel<T, VEC, PP, Z, 0, true><<<plan.blocks, plan.threads, 0, stream>>>(p);
      else
        return cudaErrorInvalidConfiguration;
    }
    return cudaGetLastError();
  });
}

}  // namespace gdn

using namespace gdn;

extern "C" {

gdn_status_t group_norm_fwd(const group_norm_args *a, gdn_stream_t stream) {
  (void)set_host_error(GDN_OK, "");
  CHECK_THAT(a != nullptr, GDN_ERR_INVALID_ARG, "args is NULL");
  gdn_status_t st = check_norm(*a);
  if (st != GDN_OK) return st;
  if (a->B * (int64_t)a->T == 0) return GDN_OK;
  CHECK_TOKENS(a->y, "y", a->dtype);
  CHECK_THAT(a->y_stride >= a->D, GDN_ERR_INVALID_ARG, "a token stride is less than its row");
  NormParams p = norm_params(*a);
  const bool bf16 = a->dtype == GDN_BF16;
  p.y = a->y;
  p.ys = a->T > 1 ? a->y_stride : a->D;
  p.yb = a->B > 1 ? a->y_batch_stride : 0;
  p.flat = p.flat || (evenly(p, p.xs, p.xb) && (p.z == nullptr || evenly(p, p.zs, p.zb)) &&
                      evenly(p, p.ys, p.yb));
  const int vec = norm_vec(p, bf16, {p.x, p.z, p.y}, {p.xs, p.xb, p.zs, p.zb, p.ys, p.yb});
  const NormPlan plan = norm_plan(p, bf16, vec, false);
  p.err = device_error_word();
  if (p.err == nullptr) return launch_status(cudaGetLastError(), "device error word");
  return launch_status(launch_norm_fwd(p, bf16, plan, reinterpret_cast<cudaStream_t>(stream)),
                       "norm launch");
}

gdn_status_t group_norm_bwd_workspace_size(const group_norm_bwd_args *a, size_t *bytes) {
  CHECK_THAT(a != nullptr && bytes != nullptr, GDN_ERR_INVALID_ARG, "NULL argument");
  *bytes = 0;
  gdn_status_t st = check_bwd(*a);
  if (st != GDN_OK) return st;
  NormParams p = norm_params(*a);
  *bytes = bwd_workspace(*a, p, bwd_plan(*a, p));
  return GDN_OK;
}

gdn_status_t group_norm_bwd(const group_norm_bwd_args *a, gdn_stream_t stream) {
  (void)set_host_error(GDN_OK, "");
  CHECK_THAT(a != nullptr, GDN_ERR_INVALID_ARG, "args is NULL");
  gdn_status_t st = check_bwd(*a);
  if (st != GDN_OK) return st;
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  NormParams p = norm_params(*a);
  if (p.tokens == 0) {  // sums over no tokens
    const size_t n = (size_t)part_columns(p) * sizeof(float);
    cudaError_t e = cudaSuccess;
    if (a->dweight != nullptr) e = cudaMemsetAsync(a->dweight, 0, n, s);
    if (e == cudaSuccess && a->dbias != nullptr) e = cudaMemsetAsync(a->dbias, 0, n, s);
    return launch_status(e, "norm sums");
  }
  const NormPlan plan = bwd_plan(*a, p);
  const size_t need = bwd_workspace(*a, p, plan);
  if (need > 0) {
    CHECK_THAT(a->workspace != nullptr && a->workspace_bytes >= need, GDN_ERR_WORKSPACE,
               "workspace of %zu bytes needed (got %zu)", need, a->workspace_bytes);
    CHECK_PTR(a->workspace, "workspace");
    p.part = static_cast<float *>(a->workspace);
  }
  p.err = device_error_word();
  if (p.err == nullptr) return launch_status(cudaGetLastError(), "device error word");
  cudaError_t e = launch_norm_bwd(p, a->dtype == GDN_BF16, plan, s);
  if (e == cudaSuccess && need > 0)
    e = launch_norm_sums(p.part, part_rows(p, plan), part_columns(p), a->dweight, a->dbias, s);
  return launch_status(e, "norm gradient launch");
}

}  // extern "C"
