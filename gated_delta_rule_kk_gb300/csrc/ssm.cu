// C entry points of the state space scan, and its form for single tokens.
//
// ssm_decode streams each request's state [V, K] once through registers: a row
// of K elements lies over 8, 16 or 32 lanes in 16-byte pieces, a thread holds
// the pieces of 8 rows (all on the way at once), takes the T tokens in float32
// and writes the rows back.  The bytes of the state, read and written once,
// bound it; a block is one head of one request, with no shared memory and no
// barrier, so that many of them hide the trip to memory.
#include <math.h>

#include "abi_check.h"
#include "rows.cuh"
#include "ssm_items.cuh"

namespace gdn {
namespace {

constexpr int SD_ROWS = 8;   // state rows of a thread
constexpr int SD_WARPS = 4;

struct SsmDecodeParams {
  const void *x, *z, *Bm, *Cm, *dt;
  const float *A_log, *D, *dt_bias;
  void *state, *y;
  const int32_t *slots;
  int *err;
  int64_t xs, xb, zs, zb, bs, bb, cs, cb, dts, dtb, ys, yb;
  int B, T, H, Hg, K, V, pool;
  int dt_f32, softplus, y_f32;
  int tok_f32;   // type of x, z, Bm, Cm
  int whole_bc;  // rows of Bm and Cm are read in 16-byte pieces
  int vblocks;
};

// VEC values of a row of B or C from column k on
template <typename T, int VEC>
__device__ __forceinline__ void load_bc(float *f, const T *row, bool whole) {
  if (whole) {
    constexpr int PIECE = VEC * sizeof(T) > 16 ? 16 / (int)sizeof(T) : VEC;
#pragma unroll
    for (int i = 0; i < VEC; i += PIECE) {
      Row<T, PIECE> r;
      r.load(row + i);
      r.widen(f + i);
    }
  } else {
#pragma unroll
    for (int i = 0; i < VEC; ++i) f[i] = to_f32(row[i]);
  }
}

// e^x to the rounding of the plain exponential, products and sums rounded one by
// one below: a bfloat16 state is rounded again at every call, so two ways of
// writing the same update would drift apart a unit at a time.
//
// The T tokens are taken as one small chunk.  With G_t the decays' running sum
// and u_t = s_t x_t,
//   y_t = e^(G_t) (h C_t) + sum_{s<=t} e^(G_t - G_s) (B_s . C_t) u_s
//   h  <- e^(G_T) h + sum_t (u_t e^(G_T - G_t)) B_t^T
// so the state is met with 2 T + 2 operations an element instead of 3 T, once
// for all tokens.
//
// S: type of the state; LPR: lanes of a row; PP: pieces of a lane (K <= LPR *
// PP * VEC); TM: tokens, or more.  grid: (request, head, block of rows).
template <typename S, int LPR, int PP, int TM>
__global__ void __launch_bounds__(32 * SD_WARPS) ssm_decode_kernel(SsmDecodeParams p) {
  constexpr int VEC = 16 / (int)sizeof(S), RPS = 32 / LPR;  // rows of a warp at a time
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int64_t bh = blockIdx.x / p.vblocks;
  const int b = (int)(bh / p.H), h = (int)(bh % p.H), g = h / (p.H / p.Hg);
  if (!bounds_ok(b < p.B && h < p.H && g < p.Hg, p.err)) return;
  const int v0 = ((blockIdx.x % p.vblocks) * SD_WARPS + warp) * SD_ROWS * RPS + lane / LPR;
  const int k0 = (lane % LPR) * VEC, K = p.K, V = p.V;
  const int slot = p.slots ? p.slots[b] : b;
  auto row = [&](int j) { return v0 + j * RPS; };
  // the sum of row j over its lanes ends in the lanes whose high bits are j
  const int vown = row((lane % LPR) / (LPR / SD_ROWS));
  const bool writes = lane % (LPR / SD_ROWS) == 0 && vown < V;
  auto put = [&](int t, float y) {
    const int64_t at = b * p.yb + t * p.ys + (int64_t)h * V + vown;
    if (p.y_f32)
      static_cast<float *>(p.y)[at] = y;
    else
      static_cast<__nv_bfloat16 *>(p.y)[at] = __float2bfloat16_rn(y);
  };
  if (slot < 0 || slot >= p.pool) {
    if (threadIdx.x == 0) record_error(p.err, GDN_ERR_BAD_SLOT);
    if (writes)
      for (int t = 0; t < p.T; ++t) put(t, 0.f);
    return;
  }
  S *state = static_cast<S *>(p.state) + ((int64_t)slot * p.H + h) * V * K + k0;
  Row<S, VEC> raw[SD_ROWS][PP];
#pragma unroll
  for (int j = 0; j < SD_ROWS; ++j)
#pragma unroll
    for (int q = 0; q < PP; ++q) {
      if (row(j) < V && k0 + q * LPR * VEC < K)
        raw[j][q].load(state + (int64_t)row(j) * K + q * LPR * VEC);
      else
        raw[j][q].zero();
    }
  auto token = [&](const void *base, int64_t at) {
    return p.tok_f32 ? static_cast<const float *>(base)[at]
                     : to_f32(static_cast<const __nv_bfloat16 *>(base)[at]);
  };
  auto pieces = [&](float *f, const void *base, int64_t at, int q) {
    at += k0 + q * LPR * VEC;
    if (k0 + q * LPR * VEC >= K) {
#pragma unroll
      for (int e = 0; e < VEC; ++e) f[e] = 0.f;
    } else if (p.tok_f32) {
      load_bc<float, VEC>(f, static_cast<const float *>(base) + at, p.whole_bc);
    } else {
      load_bc<__nv_bfloat16, VEC>(f, static_cast<const __nv_bfloat16 *>(base) + at, p.whole_bc);
    }
  };
  const int64_t xat = b * p.xb + (int64_t)h * V, bat = b * p.bb + (int64_t)g * K;
  const int64_t cat = b * p.cb + (int64_t)g * K;
  const float a = -expf(p.A_log[h]), bias = p.dt_bias ? p.dt_bias[h] : 0.f;
  float step[TM], G[TM], xown[TM], total = 0.f;
#pragma unroll
  for (int t = 0; t < TM; ++t) {
    step[t] = xown[t] = 0.f;
    if (t < p.T) {
      step[t] = ssm_step(p, b * p.dtb + t * p.dts, h, bias);
      total = __fadd_rn(total, __fmul_rn(a, step[t]));
      if (vown < V) xown[t] = token(p.x, xat + t * p.xs + vown);
    }
    G[t] = total;
  }
  float s[SD_ROWS][PP][VEC];
#pragma unroll
  for (int j = 0; j < SD_ROWS; ++j)
#pragma unroll
    for (int q = 0; q < PP; ++q) raw[j][q].widen(s[j][q]);
#pragma unroll
  for (int t = 0; t < TM; ++t) {
    if (t >= p.T) break;
    float sum[SD_ROWS] = {}, dots[TM] = {};
#pragma unroll
    for (int q = 0; q < PP; ++q) {
      float cv[VEC];
      pieces(cv, p.Cm, cat + t * p.cs, q);
#pragma unroll
      for (int j = 0; j < SD_ROWS; ++j) {
        float acc[2] = {0.f, 0.f};
#pragma unroll
        for (int e = 0; e < VEC; e += 2) fma_row<2>(acc, s[j][q] + e, cv + e);
        sum[j] += acc[0] + acc[1];
      }
#pragma unroll
      for (int r = 0; r <= t; ++r) {
        float bv[VEC], acc[2] = {0.f, 0.f};
        pieces(bv, p.Bm, bat + r * p.bs, q);
#pragma unroll
        for (int e = 0; e < VEC; e += 2) fma_row<2>(acc, bv + e, cv + e);
        dots[r] += acc[0] + acc[1];
      }
    }
    // halve the rows and the lanes of a row at each step, then the lanes alone
#pragma unroll
    for (int n = SD_ROWS / 2, o = LPR / 2; o > 0; n /= 2, o /= 2) {
      if (n > 0) {
        const bool up = lane & o;
#pragma unroll
        for (int j = 0; j < n; ++j) {
          const float send = up ? sum[j] : sum[j + n], keep = up ? sum[j + n] : sum[j];
          sum[j] = keep + __shfl_xor_sync(~0u, send, o);
        }
      } else {
        sum[0] += __shfl_xor_sync(~0u, sum[0], o);
      }
#pragma unroll
      for (int r = 0; r <= t; ++r) dots[r] += __shfl_xor_sync(~0u, dots[r], o);
    }
    if (!writes) continue;
    float y = expf(G[t]) * sum[0];
#pragma unroll
    for (int r = 0; r <= t; ++r) y = fmaf(expf(G[t] - G[r]) * dots[r], step[r] * xown[r], y);
    if (p.D) y = fmaf(p.D[h], xown[t], y);
    if (p.z) y *= silu(token(p.z, b * p.zb + t * p.zs + (int64_t)h * V + vown));
    put(t, y);
  }
  const float keep = expf(total);
  float w[TM][SD_ROWS];
#pragma unroll
  for (int t = 0; t < TM; ++t) {
    const float e = expf(total - G[t]);
#pragma unroll
    for (int j = 0; j < SD_ROWS; ++j)
      w[t][j] = t < p.T && row(j) < V
                    ? __fmul_rn(__fmul_rn(token(p.x, xat + t * p.xs + row(j)), step[t]), e)
                    : 0.f;
  }
#pragma unroll
  for (int q = 0; q < PP; ++q) {
    float bv[TM][VEC];
#pragma unroll
    for (int t = 0; t < TM; ++t)
      if (t < p.T)
        pieces(bv[t], p.Bm, bat + t * p.bs, q);
      else
#pragma unroll
        for (int e = 0; e < VEC; ++e) bv[t][e] = 0.f;
    if (k0 + q * LPR * VEC >= K) continue;
#pragma unroll
    for (int j = 0; j < SD_ROWS; ++j) {
      if (row(j) >= V) continue;
      float out[VEC];
#pragma unroll
      for (int e = 0; e < VEC; ++e) {
        float add = __fmul_rn(w[0][j], bv[0][e]);
#pragma unroll
        for (int t = 1; t < TM; ++t) add = __fmaf_rn(w[t][j], bv[t][e], add);
        out[e] = __fadd_rn(__fmul_rn(keep, s[j][q][e]), add);
      }
      Row<S, VEC> r;
      r.round(out);
      r.store(state + (int64_t)row(j) * K + q * LPR * VEC);
    }
  }
}

template <typename S, int LPR, int PP>
void launch_tokens(const SsmDecodeParams &p, unsigned grid, cudaStream_t stream) {
  if (p.T == 1)
    ssm_decode_kernel<S, LPR, PP, 1><<<grid, 32 * SD_WARPS, 0, stream>>>(p);
  else if (p.T == 2)
    ssm_decode_kernel<S, LPR, PP, 2><<<grid, 32 * SD_WARPS, 0, stream>>>(p);
  else
    ssm_decode_kernel<S, LPR, PP, 4><<<grid, 32 * SD_WARPS, 0, stream>>>(p);
}

template <typename S>
cudaError_t launch_decode(SsmDecodeParams &p, int64_t bh, cudaStream_t stream) {
  const int pieces = p.K * (int)sizeof(S) / 16;
  const int lpr = pieces <= 8 ? 8 : pieces <= 16 ? 16 : 32;
  const int rows = SD_WARPS * SD_ROWS * 32 / lpr;
  p.vblocks = (p.V + rows - 1) / rows;
  const unsigned grid = (unsigned)(bh * p.vblocks);
  if (lpr == 8)
    launch_tokens<S, 8, 1>(p, grid, stream);
  else if (lpr == 16)
    launch_tokens<S, 16, 1>(p, grid, stream);
  else if (pieces <= 32)
    launch_tokens<S, 32, 1>(p, grid, stream);
  else
    launch_tokens<S, 32, 2>(p, grid, stream);
  return cudaGetLastError();
}

// Checks shared by the two forms.
template <typename Args>
gdn_status_t check_ssm(const Args &a) {
  CHECK_DTYPE(a.dtype, "dtype");
  CHECK_DTYPE(a.dt_dtype, "dt_dtype");
  CHECK_THAT(a.dt_dtype == GDN_F32 || a.dt_dtype == a.dtype, GDN_ERR_INVALID_ARG,
             "dt_dtype must be GDN_F32 or dtype");
  CHECK_THAT(a.B >= 1 && a.T >= 0 && a.H >= 1 && a.Hg >= 1 && a.K >= 1 && a.V >= 1,
             GDN_ERR_INVALID_ARG, "sizes must be positive (B=%d T=%d heads=%d/%d K=%d V=%d)", a.B,
             a.T, a.Hg, a.H, a.K, a.V);
  CHECK_THAT(a.H % a.Hg == 0, GDN_ERR_UNSUPPORTED, "H (%d) must be a multiple of Hg (%d)", a.H, a.Hg);
  CHECK_THAT(a.H <= MAX_GRID_YZ, GDN_ERR_UNSUPPORTED, "H (%d) must be at most %d", a.H, MAX_GRID_YZ);
  CHECK_THAT(a.K <= 256, GDN_ERR_UNSUPPORTED, "K=%d exceeds 256", a.K);
  CHECK_FLAG(a.dt_softplus, "dt_softplus");
  CHECK_FLAG(a.y_fp32, "y_fp32");
  if (a.T > 0) {
    CHECK_TOKENS(a.x, "x", a.dtype);
    if (a.z != nullptr) CHECK_TOKENS(a.z, "z", a.dtype);
    CHECK_TOKENS(a.Bm, "Bm", a.dtype);
    CHECK_TOKENS(a.Cm, "Cm", a.dtype);
    CHECK_TOKENS(a.y, "y", a.y_fp32 ? GDN_F32 : a.dtype);
    CHECK_TOKENS(a.dt, "dt", a.dt_dtype);
    const int64_t hv = (int64_t)a.H * a.V, gk = (int64_t)a.Hg * a.K;
    CHECK_THAT(a.x_stride >= hv && a.y_stride >= hv && (a.z == nullptr || a.z_stride >= hv) &&
                   a.Bm_stride >= gk && a.Cm_stride >= gk && a.dt_stride >= a.H,
               GDN_ERR_INVALID_ARG, "a token stride is less than its row");
  }
  CHECK_PTR(a.A_log, "A_log");
  CHECK_OPT_PTR(a.D, "D");
  CHECK_OPT_PTR(a.dt_bias, "dt_bias");
  return GDN_OK;
}

// Copies what both forms' parameters share.
template <typename P, typename Args>
void set_tokens(P &p, const Args &a) {
  p.x = a.x; p.z = a.z; p.Bm = a.Bm; p.Cm = a.Cm; p.dt = a.dt;
  p.A_log = a.A_log; p.D = a.D; p.dt_bias = a.dt_bias; p.y = a.y;
  const bool many = a.B > 1;
  p.xs = a.x_stride; p.xb = many ? a.x_batch_stride : 0;
  p.zs = a.z_stride; p.zb = many ? a.z_batch_stride : 0;
  p.bs = a.Bm_stride; p.bb = many ? a.Bm_batch_stride : 0;
  p.cs = a.Cm_stride; p.cb = many ? a.Cm_batch_stride : 0;
  p.dts = a.dt_stride; p.dtb = many ? a.dt_batch_stride : 0;
  p.ys = a.y_stride; p.yb = many ? a.y_batch_stride : 0;
  p.B = a.B; p.T = a.T; p.H = a.H; p.Hg = a.Hg; p.K = a.K; p.V = a.V;
  p.dt_f32 = a.dt_dtype == GDN_F32;
  p.softplus = a.dt_softplus;
  p.y_f32 = a.y_fp32 || a.dtype == GDN_F32;
}

gdn_status_t check_chunk_args(const ssm_chunk_args &a) {
  gdn_status_t st = check_ssm(a);
  if (st != GDN_OK) return st;
  CHECK_THAT(a.N >= 1 && a.N <= MAX_GRID_YZ, GDN_ERR_UNSUPPORTED, "N (%d) must be in 1..%d", a.N,
             MAX_GRID_YZ);
  CHECK_THAT(a.V <= 32 * MAX_GRID_YZ, GDN_ERR_UNSUPPORTED, "V (%d) must be at most %d", a.V,
             32 * MAX_GRID_YZ);
  CHECK_THAT(a.segment_tokens >= 0 && a.segment_tokens % SSM_UNIT == 0, GDN_ERR_INVALID_ARG,
             "segment_tokens (%d) must be 0 or a multiple of %d", a.segment_tokens, SSM_UNIT);
  if (a.cu_seqlens == nullptr) {
    CHECK_THAT(a.N == a.B, GDN_ERR_INVALID_ARG, "without cu_seqlens N (%d) must equal B (%d)", a.N,
               a.B);
  } else {
    CHECK_THAT(a.B == 1, GDN_ERR_INVALID_ARG, "with cu_seqlens B must be 1 (got %d)", a.B);
    CHECK_OPT_PTR(a.cu_seqlens, "cu_seqlens");
  }
  CHECK_OPT_PTR(a.h0, "h0");
  CHECK_OPT_PTR(a.ht, "ht");
  return GDN_OK;
}

// Segment length when the caller leaves it open.  Cutting costs a second pass
// over x, B and dt and a block reads the states of the segments before its own,
// so sequences stay whole when they give half the blocks the GPU holds; else
// segments are as long as still fills it, at most 64 to a sequence.
int choose_segment(const SsmParams &p, bool tc) {
  const int cols = tc ? 64 : 32;  // of a block's state tile; one block an SM, or four
  const int64_t chains = (int64_t)p.H * ((p.V + cols - 1) / cols);
  const int64_t want = (tc ? 1 : 4) * (int64_t)sm_count();
  if (p.cu == nullptr && chains * p.N >= want / 2) return SSM_WHOLE;
  const int64_t tokens = p.cu ? p.T : (int64_t)p.T * p.N;
  int64_t seg = tokens * chains / want;
  if (seg < p.T / 64) seg = p.T / 64;
  seg = (seg + SSM_UNIT - 1) / SSM_UNIT * SSM_UNIT;
  return seg < SSM_UNIT ? SSM_UNIT : seg < p.T ? (int)seg : SSM_WHOLE;
}

SsmParams chunk_params(const ssm_chunk_args &a) {
  SsmParams p{};
  set_tokens(p, a);
  p.N = a.N;
  p.h0 = a.h0; p.ht = a.ht; p.cu = a.cu_seqlens;
  p.seg = a.segment_tokens > 0 ? a.segment_tokens
                               : choose_segment(p, ssm_tc_supported(p, a.dtype == GDN_BF16));
  const int64_t longest = a.T;  // no sequence has more tokens
  const int64_t per = longest > p.seg ? (longest + p.seg - 1) / p.seg : 1;
  p.items = (int)(a.cu_seqlens ? (a.N + (longest > p.seg ? longest / p.seg : 0)) : a.N * per);
  return p;
}

// Workspace: segment states, then their decays.  None if no sequence is cut.
size_t chunk_workspace(const SsmParams &p) {
  if (p.T <= p.seg) return 0;
  const size_t states = (size_t)p.items * p.H * p.V * p.K * sizeof(float);
  return states + (size_t)p.items * p.H * sizeof(float);
}

}  // namespace
}  // namespace gdn

using namespace gdn;

extern "C" {

gdn_status_t ssm_chunk_workspace_size(const ssm_chunk_args *a, size_t *bytes) {
  CHECK_THAT(a != nullptr && bytes != nullptr, GDN_ERR_INVALID_ARG, "NULL argument");
  *bytes = 0;
  gdn_status_t st = check_chunk_args(*a);
  if (st != GDN_OK) return st;
  *bytes = chunk_workspace(chunk_params(*a));
  return GDN_OK;
}

gdn_status_t ssm_chunk_fwd(const ssm_chunk_args *a, gdn_stream_t stream) {
  (void)set_host_error(GDN_OK, "");
  CHECK_THAT(a != nullptr, GDN_ERR_INVALID_ARG, "args is NULL");
  gdn_status_t st = check_chunk_args(*a);
  if (st != GDN_OK) return st;
  SsmParams p = chunk_params(*a);
  const size_t need = chunk_workspace(p);
  if (need > 0) {
    CHECK_THAT(a->workspace != nullptr && a->workspace_bytes >= need, GDN_ERR_WORKSPACE,
               "workspace of %zu bytes needed (got %zu)", need, a->workspace_bytes);
    CHECK_THAT(aligned_to(a->workspace, 256), GDN_ERR_MISALIGNED,
               "workspace is not 256-byte aligned");
    p.seg_state = static_cast<float *>(a->workspace);
    p.seg_decay = p.seg_state + (size_t)p.items * p.H * p.V * p.K;
  }
  p.err = device_error_word();
  if (p.err == nullptr) return launch_status(cudaGetLastError(), "device error word");
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  const bool bf16 = a->dtype == GDN_BF16;
  return launch_status(ssm_tc_supported(p, bf16) ? launch_ssm_tc(p, s) : launch_ssm_simt(p, bf16, s),
                       "scan launch");
}

gdn_status_t ssm_decode(const ssm_decode_args *a, gdn_stream_t stream) {
  (void)set_host_error(GDN_OK, "");
  CHECK_THAT(a != nullptr, GDN_ERR_INVALID_ARG, "args is NULL");
  CHECK_THAT(a->T >= 1 && a->T <= 4, GDN_ERR_UNSUPPORTED, "T must be 1..4 (got %d)", a->T);
  gdn_status_t st = check_ssm(*a);
  if (st != GDN_OK) return st;
  CHECK_DTYPE(a->state_dtype, "state_dtype");
  CHECK_THAT(a->K % 8 == 0, GDN_ERR_UNSUPPORTED, "K (%d) must be a multiple of 8", a->K);
  CHECK_THAT(a->pool >= 1, GDN_ERR_INVALID_ARG, "pool must be positive (got %d)", a->pool);
  CHECK_THAT(a->slot_indices != nullptr || a->pool >= a->B, GDN_ERR_INVALID_ARG,
             "identity slots need pool (%d) >= B (%d)", a->pool, a->B);
  CHECK_PTR(a->state, "state");
  CHECK_OPT_PTR(a->slot_indices, "slot_indices");
  const int64_t bh = (int64_t)a->B * a->H;
  CHECK_THAT(bh * ((a->V + 15) / 16) <= 0x7fffffff, GDN_ERR_UNSUPPORTED,
             "B * H (%lld) is too large for one call", (long long)bh);
  SsmDecodeParams p{};
  set_tokens(p, *a);
  p.state = a->state; p.slots = a->slot_indices; p.pool = a->pool;
  const int wide = 16 / (int)dtype_bytes(a->dtype);
  p.whole_bc = aligned_to(a->Bm, 16) && aligned_to(a->Cm, 16) && p.bs % wide == 0 && p.bb % wide == 0 && p.cs % wide == 0 && p.cb % wide == 0;
  p.err = device_error_word();
  if (p.err == nullptr) return launch_status(cudaGetLastError(), "device error word");
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  p.tok_f32 = a->dtype == GDN_F32;
  const cudaError_t e = a->state_dtype == GDN_BF16 ? launch_decode<__nv_bfloat16>(p, bh, s)
                                                   : launch_decode<float>(p, bh, s);
  return launch_status(e, "scan token launch");
}

}  // extern "C"
