// C entry points of the state space scan, and its form for single tokens.
//
// ssm_decode streams each request's state [V, K] once through registers: a row
// of K elements lies over 8, 16 or 32 lanes in 16-byte pieces, a thread holds
// the pieces of 8 rows, takes the T tokens in float32 and writes the rows back.
// The bytes of the state, read and written once, bound it.  Two kernels share
// that code:
//   few items (one head of one request, some rows of it): a block each, rows
//   from global memory straight to registers, all on the way at once; no barrier
//   and no shared memory, for the shortest call;
//   many: persistent blocks, whose items stream through a ring of bulk copies
//   in shared memory, loads several items ahead and stores behind, while other
//   warps turn the items' tokens into float32 coefficients beside the tiles, so
//   that memory never waits for a block's start, its arithmetic or its end and
//   the warps that hold the state wait for nothing but shared memory.
// Measured: one token of 256 requests, 64 heads, bf16 states of 64 x 128 93.1 us,
// 5.8 TB/s (86% of the copy rate); four tokens of 3 requests, 48 heads, float32
// states 9.4 us: the trip to memory for the states, then the tokens one after another,
// whose rows of B and C (asked for ahead only for a single token) come between the
// sums over K.
#include <math.h>

#include <algorithm>
#include <cmath>

#include "abi_check.h"
#include "ptx.cuh"
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
  float none;    // -0
  int vblocks, rows;  // blocks of rows of a head; rows of a ring tile
};

// e^x to the rounding of the plain exponential, products and sums rounded one by
// one below: a bfloat16 state is rounded again at every call, so two ways of
// writing the same update would drift apart a unit at a time.  (A product is taken
// as a x b + (-0), with a -0 that the compiler does not know: it fuses a packed
// multiplication with the addition behind it.)
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
struct SdItem {
  int b, h, slot;
  int v, end;  // rows v .. end - 1
};

// The log-decays after token r up to token t, from the tokens' own: no difference of
// running sums, of which little is left after a token that resets the state.
template <int TM>
__device__ __forceinline__ float decay_between(const float (&g)[TM], int r, int t) {
  float sum = 0.f;
#pragma unroll
  for (int q = 1; q < TM; ++q)
    if (q > r && q <= t) sum = __fadd_rn(sum, g[q]);
  return sum;
}

// What a thread needs of an item's tokens, asked for before the item's state is
// waited for.  Raw bits, so that nothing waits for them either; B and C of one
// token (of more they are read where they are used).
template <int VEC, int PP, int TM>
struct SdTokens {
  static constexpr bool BC = TM == 1;
  uint32_t b[PP][VEC], c[PP][VEC];
  uint32_t x[TM][SD_ROWS], xown[TM], zown[TM], dt[TM];
  float A_log, bias, skip;
};

template <typename S, int LPR, int PP, int TM>
struct SdRows {
  static constexpr int VEC = 16 / (int)sizeof(S), RPS = 32 / LPR;  // rows of a warp at a time
  const SsmDecodeParams *pp;
  SdItem it;
  int v0, k0, vown;
  bool writes;
  int64_t xat, bat, cat;
  SdTokens<VEC, PP, TM> tok;

  // rows it.v + warp_rows + lane / LPR + j RPS of the item
  __device__ __forceinline__ SdRows(const SsmDecodeParams &p, const SdItem &it_, int warp_rows)
      : pp(&p), it(it_) {
    const int lane = threadIdx.x & 31, g = it.h / (p.H / p.Hg);
    v0 = it.v + warp_rows + lane / LPR;
    k0 = (lane % LPR) * VEC;
    // the sum of row j over its lanes ends in the lanes whose high bits are j
    vown = row((lane % LPR) / (LPR / SD_ROWS));
    writes = lane % (LPR / SD_ROWS) == 0 && vown < it.end;
    xat = it.b * p.xb + (int64_t)it.h * p.V;
    bat = it.b * p.bb + (int64_t)g * p.K;
    cat = it.b * p.cb + (int64_t)g * p.K;
  }
  __device__ __forceinline__ int row(int j) const { return v0 + j * RPS; }
  __device__ __forceinline__ bool good() const {
    const SsmDecodeParams &p = *pp; return it.slot >= 0 && it.slot < p.pool; }
  __device__ __forceinline__ uint32_t bits(const void *base, int64_t at) const {
    const SsmDecodeParams &p = *pp;
    return p.tok_f32 ? static_cast<const uint32_t *>(base)[at]
                     : (uint32_t) static_cast<const uint16_t *>(base)[at];
  }
  __device__ __forceinline__ float value(uint32_t w) const {
    const SsmDecodeParams &p = *pp;
    return __uint_as_float(p.tok_f32 ? w : w << 16);
  }
  // VEC values of a row of B or C from this lane's column of piece q on: as raw
  // bits (bf16 pairs in the first half), and widened
  __device__ __forceinline__ void raw_pieces(uint32_t (&w)[VEC], const void *base, int64_t at,
                                             int q) const {
    const SsmDecodeParams &p = *pp;
    at += k0 + q * LPR * VEC;
#pragma unroll
    for (int e = 0; e < VEC; ++e) w[e] = 0;
    if (k0 + q * LPR * VEC >= p.K) return;
    if (p.tok_f32) {
      const uint32_t *src = static_cast<const uint32_t *>(base) + at;
      if (p.whole_bc) {
#pragma unroll
        for (int e = 0; e < VEC; e += 4) {
          const uint4 u = *reinterpret_cast<const uint4 *>(src + e);
          w[e] = u.x; w[e + 1] = u.y; w[e + 2] = u.z; w[e + 3] = u.w;
        }
      } else {
#pragma unroll
        for (int e = 0; e < VEC; ++e) w[e] = src[e];
      }
    } else {
      const uint16_t *src = static_cast<const uint16_t *>(base) + at;
      if (p.whole_bc) {
#pragma unroll
        for (int e = 0; e < VEC / 2; e += 2) {
          const uint2 u = *reinterpret_cast<const uint2 *>(src + 2 * e);
          w[e] = u.x; w[e + 1] = u.y;
        }
      } else {
#pragma unroll
        for (int e = 0; e < VEC / 2; ++e) w[e] = src[2 * e] | (uint32_t)src[2 * e + 1] << 16;
      }
    }
  }
  __device__ __forceinline__ void widen(float *f, const uint32_t (&w)[VEC]) const {
    const SsmDecodeParams &p = *pp;
#pragma unroll
    for (int e = 0; e < VEC / 2; ++e) {
      f[2 * e] = __uint_as_float(p.tok_f32 ? w[2 * e] : w[e] << 16);
      f[2 * e + 1] = __uint_as_float(p.tok_f32 ? w[2 * e + 1] : w[e] & 0xffff0000u);
    }
  }

  __device__ __forceinline__ void fetch() {
    const SsmDecodeParams &p = *pp;
    tok.A_log = p.A_log[it.h];
    tok.bias = p.dt_bias ? p.dt_bias[it.h] : 0.f;
    tok.skip = p.D ? p.D[it.h] : 0.f;
#pragma unroll
    for (int t = 0; t < TM; ++t) {
      tok.dt[t] = tok.xown[t] = tok.zown[t] = 0;
      if (t < p.T) {
        const int64_t dat = it.b * p.dtb + t * p.dts + it.h;
        tok.dt[t] = p.dt_f32 ? static_cast<const uint32_t *>(p.dt)[dat]
                             : (uint32_t) static_cast<const uint16_t *>(p.dt)[dat];
        if (vown < it.end) {
          tok.xown[t] = bits(p.x, xat + t * p.xs + vown);
          if (p.z) tok.zown[t] = bits(p.z, it.b * p.zb + t * p.zs + (int64_t)it.h * p.V + vown);
        }
      }
#pragma unroll
      for (int j = 0; j < SD_ROWS; ++j)
        tok.x[t][j] = t < p.T && row(j) < it.end ? bits(p.x, xat + t * p.xs + row(j)) : 0;
    }
    if (tok.BC) {
#pragma unroll
      for (int q = 0; q < PP; ++q) {
        raw_pieces(tok.b[q], p.Bm, bat, q);
        raw_pieces(tok.c[q], p.Cm, cat, q);
      }
    }
  }

  __device__ __forceinline__ void pieces(float *f, bool of_b, int t, int q) const {
    const SsmDecodeParams &p = *pp;
    if (tok.BC) {
      widen(f, of_b ? tok.b[q] : tok.c[q]);
    } else {
      uint32_t w[VEC];
      if (of_b)
        raw_pieces(w, p.Bm, bat + t * p.bs, q);
      else
        raw_pieces(w, p.Cm, cat + t * p.cs, q);
      widen(f, w);
    }
  }
  __device__ __forceinline__ void put(int t, float y) const {
    const SsmDecodeParams &p = *pp;
    const int64_t at = it.b * p.yb + t * p.ys + (int64_t)it.h * p.V + vown;
    if (p.y_f32)
      static_cast<float *>(p.y)[at] = y;
    else
      static_cast<__nv_bfloat16 *>(p.y)[at] = __float2bfloat16_rn(y);
  }
  __device__ __forceinline__ void refuse() const {
    const SsmDecodeParams &p = *pp;
    if (threadIdx.x == 0) record_error(p.err, GDN_ERR_BAD_SLOT);
    if (writes)
      for (int t = 0; t < p.T; ++t) put(t, 0.f);
  }

  // The item's rows, read from `src` and written to `dst` (row it.v's first
  // element; global or shared memory).
  __device__ __forceinline__ void take(const S *src, S *dst) const {
    const SsmDecodeParams &p = *pp;
    const int lane = threadIdx.x & 31, K = p.K, end = it.end;
    Row<S, VEC> raw[SD_ROWS][PP];
#pragma unroll
    for (int j = 0; j < SD_ROWS; ++j)
#pragma unroll
      for (int q = 0; q < PP; ++q) {
        if (row(j) < end && k0 + q * LPR * VEC < K)
          raw[j][q].load(src + (row(j) - it.v) * K + k0 + q * LPR * VEC);
        else
          raw[j][q].zero();
      }
    const float a = -expf(tok.A_log);
    float step[TM], g[TM], G[TM], total = 0.f;
#pragma unroll
    for (int t = 0; t < TM; ++t) {
      step[t] = g[t] = 0.f;
      if (t < p.T) {
        const float dt = __uint_as_float(p.dt_f32 ? tok.dt[t] : tok.dt[t] << 16);
        step[t] = ssm_softplus(p, __fadd_rn(dt, tok.bias));
        g[t] = __fmul_rn(a, step[t]);
        total = __fadd_rn(total, g[t]);
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
        pieces(cv, false, t, q);
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
          pieces(bv, true, r, q);
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
      for (int r = 0; r <= t; ++r)
        y = fmaf(expf(decay_between(g, r, t)) * dots[r], step[r] * value(tok.xown[r]), y);
      if (p.D) y = fmaf(tok.skip, value(tok.xown[t]), y);
      if (p.z) y *= silu(value(tok.zown[t]));
      put(t, y);
    }
    const float keep = expf(total);
    float e[TM];
#pragma unroll
    for (int t = 0; t < TM; ++t) e[t] = expf(decay_between(g, t, TM - 1));
#pragma unroll
    for (int q = 0; q < PP; ++q) {
      float bv[TM][VEC];
#pragma unroll
      for (int t = 0; t < TM; ++t)
        if (t < p.T)
          pieces(bv[t], true, t, q);
        else
#pragma unroll
          for (int i = 0; i < VEC; ++i) bv[t][i] = 0.f;
      if (k0 + q * LPR * VEC >= K) continue;
#pragma unroll
      for (int j = 0; j < SD_ROWS; ++j) {
        if (row(j) >= end) continue;
        float w[TM], out[VEC];
#pragma unroll
        for (int t = 0; t < TM; ++t)
          w[t] = __fmul_rn(__fmul_rn(value(tok.x[t][j]), step[t]), e[t]);
#pragma unroll
        for (int i = 0; i < VEC; i += 2) {
          float add[2];
          const float w0[2] = {w[0], w[0]}, kk[2] = {keep, keep}, none[2] = {p.none, p.none};
          fma_rows<2>(add, w0, bv[0] + i, none);
#pragma unroll
          for (int t = 1; t < TM; ++t) {
            const float wt[2] = {w[t], w[t]};
            fma_row<2>(add, wt, bv[t] + i);
          }
          fma_rows<2>(out + i, kk, s[j][q] + i, none);
          add_row<2>(out + i, out + i, add);
        }
        Row<S, VEC> r;
        r.round(out);
        r.store(dst + (row(j) - it.v) * K + k0 + q * LPR * VEC);
      }
    }
  }
};

// grid: (request, head, block of SD_WARPS * SD_ROWS * RPS rows).
template <typename S, int LPR, int PP, int TM>
__global__ void __launch_bounds__(32 * SD_WARPS) ssm_decode_kernel(SsmDecodeParams p) {
  constexpr int WARP_ROWS = SD_ROWS * 32 / LPR;
  const int64_t bh = blockIdx.x / p.vblocks;
  SdItem it;
  it.b = (int)(bh / p.H);
  it.h = (int)(bh % p.H);
  it.v = (int)(blockIdx.x % p.vblocks) * SD_WARPS * WARP_ROWS;
  if (!bounds_ok(it.b < p.B && it.h < p.H && it.v < p.V, p.err)) return;
  it.end = p.V;
  it.slot = p.slots ? p.slots[it.b] : it.b;
  S *state = static_cast<S *>(p.state) + (((int64_t)it.slot * p.H + it.h) * p.V + it.v) * p.K;
  SdRows<S, LPR, PP, TM> rows(p, it, (threadIdx.x >> 5) * WARP_ROWS);
  if (!rows.good()) return rows.refuse();
  rows.fetch();
  rows.take(state, state);
}

// The ring: SD_STAGES tiles of p.rows rows, each with the item's coefficients
// beside it.  Warps: SD_WARPS that take the tiles in place, SD_PREP that form
// the coefficients (every SD_PREP-th item each), one that loads and one that
// stores tiles.  Every wait is bounded.
constexpr int SD_STAGES = 4, SD_PREP = 3;
// (a preparing warp skips SD_PREP - 1 items; it may not skip a use of a barrier)
static_assert(SD_PREP <= SD_STAGES, "barrier phases");
// blocks an SM holds (coefficients of four tokens take too many registers for 3)
constexpr int sd_blocks(int tm) { return tm > 2 ? 2 : 3; }
constexpr uint32_t SD_TILE = 16384;
constexpr int SD_THREADS = 32 * (SD_WARPS + SD_PREP + 2);

// Coefficients of an item with T tokens (floats): B and C [T][K], padded to
// whole pieces; per token and row u = s_t x_t, u e^(G_T - G_t), D x and silu(z);
// e^(G_t - G_s) (B_s . C_t); e^(G_t); e^(G_T).
struct SdCoef {
  int K, R, T;  // K padded, rows, tokens
  __host__ __device__ SdCoef(int k, int r, int t) : K((k + 7) / 8 * 8), R(r), T(t) {}
  __host__ __device__ int B(int t) const { return t * K; }
  __host__ __device__ int C(int t) const { return (T + t) * K; }
  __host__ __device__ int u(int t) const { return 2 * T * K + t * R; }
  __host__ __device__ int w(int t) const { return 2 * T * K + (T + t) * R; }
  __host__ __device__ int skip(int t) const { return 2 * T * K + (2 * T + t) * R; }
  __host__ __device__ int gate(int t) const { return 2 * T * K + (3 * T + t) * R; }
  __host__ __device__ int mix(int t, int r) const { return 2 * T * K + 4 * T * R + t * T + r; }
  __host__ __device__ int eG(int t) const { return 2 * T * K + 4 * T * R + T * T + t; }
  __host__ __device__ int keep() const { return 2 * T * K + 4 * T * R + T * T + T; }
  __host__ __device__ int bytes() const { return ((keep() + 1) * 4 + 127) / 128 * 128; }
};

// One warp forms an item's coefficients.  Up to 256 columns and p.rows rows:
// lane l takes columns and rows l, l + 32, ..
template <int TM>
__device__ __forceinline__ void ssm_decode_prepare(const SsmDecodeParams &p, const SdItem &it,
                                                   float *f) {
  const int lane = threadIdx.x & 31, group = it.h / (p.H / p.Hg);
  const SdCoef c(p.K, p.rows, p.T);
  auto token = [&](const void *base, int64_t at) {
    return p.tok_f32 ? static_cast<const float *>(base)[at]
                     : to_f32(static_cast<const __nv_bfloat16 *>(base)[at]);
  };
  const int64_t xat = it.b * p.xb + (int64_t)it.h * p.V + it.v;
  const int64_t zat = it.b * p.zb + (int64_t)it.h * p.V + it.v;
  const int64_t bat = it.b * p.bb + (int64_t)group * p.K, cat = it.b * p.cb + (int64_t)group * p.K;
  const float a = -expf(p.A_log[it.h]), bias = p.dt_bias ? p.dt_bias[it.h] : 0.f;
  const float D = p.D ? p.D[it.h] : 0.f;
  float step[TM], g[TM], G[TM], total = 0.f;
#pragma unroll
  for (int t = 0; t < TM; ++t) {
    step[t] = g[t] = 0.f;
    if (t < p.T) {
      step[t] = ssm_softplus(
          p, __fadd_rn(ssm_dt(p, it.b * p.dtb + t * p.dts + it.h), bias));
      g[t] = __fmul_rn(a, step[t]);
      total = __fadd_rn(total, g[t]);
    }
    G[t] = total;
  }
  float dots[TM][TM] = {};
  for (int k = lane; k < c.K; k += 32) {
    float b[TM], cc[TM];
#pragma unroll
    for (int t = 0; t < TM; ++t) {
      b[t] = t < p.T && k < p.K ? token(p.Bm, bat + t * p.bs + k) : 0.f;
      cc[t] = t < p.T && k < p.K ? token(p.Cm, cat + t * p.cs + k) : 0.f;
    }
#pragma unroll
    for (int t = 0; t < TM; ++t) {
      if (t < p.T) {
        f[c.B(t) + k] = b[t];
        f[c.C(t) + k] = cc[t];
      }
#pragma unroll
      for (int r = 0; r <= t; ++r) dots[t][r] = fmaf(b[r], cc[t], dots[t][r]);
    }
  }
  for (int r = lane; r < it.end - it.v; r += 32) {
#pragma unroll
    for (int t = 0; t < TM; ++t) {
      if (t >= p.T) continue;
      const float x = token(p.x, xat + t * p.xs + r);
      const float z = p.z ? token(p.z, zat + t * p.zs + r) : 0.f;
      const float u = __fmul_rn(x, step[t]);
      f[c.u(t) + r] = u;
      f[c.w(t) + r] = __fmul_rn(u, expf(decay_between(g, t, TM - 1)));
      f[c.skip(t) + r] = D * x;
      f[c.gate(t) + r] = p.z ? silu(z) : 1.f;
    }
  }
#pragma unroll
  for (int t = 0; t < TM; ++t)
#pragma unroll
    for (int r = 0; r <= t; ++r) {
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) dots[t][r] += __shfl_xor_sync(~0u, dots[t][r], o);
      if (lane == 0 && t < p.T) f[c.mix(t, r)] = expf(decay_between(g, r, t)) * dots[t][r];
    }
  if (lane == 0) {
#pragma unroll
    for (int t = 0; t < TM; ++t)
      if (t < p.T) f[c.eG(t)] = expf(G[t]);
    f[c.keep()] = expf(total);
  }
}

// One thread's part of a tile: rows warp_rows + lane / LPR + j RPS, one after
// another out of shared memory and back.
template <typename S, int LPR, int PP, int TM>
__device__ __forceinline__ void ssm_decode_tile(const SsmDecodeParams &p, const SdItem &it,
                                                int warp_rows, S *tile, const float *f) {
  constexpr int VEC = 16 / (int)sizeof(S), RPS = 32 / LPR;
  const int lane = threadIdx.x & 31, rows = it.end - it.v, K = p.K;
  const SdCoef c(K, p.rows, p.T);
  const int r0 = warp_rows + lane / LPR, k0 = (lane % LPR) * VEC;
  const int own = r0 + ((lane % LPR) / (LPR / SD_ROWS)) * RPS;
  const bool writes = lane % (LPR / SD_ROWS) == 0 && own < rows;
  const float keep = f[c.keep()];
  const float kk[2] = {keep, keep}, none[2] = {p.none, p.none};
  float sum[TM][SD_ROWS];
#pragma unroll
  for (int t = 0; t < TM; ++t)
#pragma unroll
    for (int j = 0; j < SD_ROWS; ++j) sum[t][j] = 0.f;
#pragma unroll
  for (int q = 0; q < PP; ++q) {
    const int k = k0 + q * LPR * VEC;
    if (k >= K) continue;
    float b[TM][VEC], cc[TM][VEC];
#pragma unroll
    for (int t = 0; t < TM; ++t)
#pragma unroll
      for (int e = 0; e < VEC; e += 4) {
        float4 u = make_float4(0.f, 0.f, 0.f, 0.f), v = u;
        if (t < p.T) {
          u = *reinterpret_cast<const float4 *>(f + c.B(t) + k + e);
          v = *reinterpret_cast<const float4 *>(f + c.C(t) + k + e);
        }
        b[t][e] = u.x; b[t][e + 1] = u.y; b[t][e + 2] = u.z; b[t][e + 3] = u.w;
        cc[t][e] = v.x; cc[t][e + 1] = v.y; cc[t][e + 2] = v.z; cc[t][e + 3] = v.w;
      }
#pragma unroll
    for (int j = 0; j < SD_ROWS; ++j) {
      const int r = r0 + j * RPS;
      if (r >= rows) continue;
      S *at = tile + r * K + k;
      Row<S, VEC> row;
      row.load(at);
      float s[VEC], out[VEC];
      row.widen(s);
#pragma unroll
      for (int t = 0; t < TM; ++t) {
        float acc[2] = {0.f, 0.f};
#pragma unroll
        for (int e = 0; e < VEC; e += 2) fma_row<2>(acc, s + e, cc[t] + e);
        sum[t][j] += acc[0] + acc[1];
      }
      float w[TM];
#pragma unroll
      for (int t = 0; t < TM; ++t) w[t] = t < p.T ? f[c.w(t) + r] : 0.f;
#pragma unroll
      for (int e = 0; e < VEC; e += 2) {
        float add[2];
        const float w0[2] = {w[0], w[0]};
        fma_rows<2>(add, w0, b[0] + e, none);
#pragma unroll
        for (int t = 1; t < TM; ++t) {
          const float wt[2] = {w[t], w[t]};
          fma_row<2>(add, wt, b[t] + e);
        }
        fma_rows<2>(out + e, kk, s + e, none);
        add_row<2>(out + e, out + e, add);
      }
      row.round(out);
      row.store(at);
    }
  }
#pragma unroll
  for (int t = 0; t < TM; ++t) {
    if (t >= p.T) break;
    // halve the rows and the lanes of a row at each step, then the lanes alone
#pragma unroll
    for (int n = SD_ROWS / 2, o = LPR / 2; o > 0; n /= 2, o /= 2) {
      if (n > 0) {
        const bool up = lane & o;
#pragma unroll
        for (int j = 0; j < n; ++j) {
          const float send = up ? sum[t][j] : sum[t][j + n], mine = up ? sum[t][j + n] : sum[t][j];
          sum[t][j] = mine + __shfl_xor_sync(~0u, send, o);
        }
      } else {
        sum[t][0] += __shfl_xor_sync(~0u, sum[t][0], o);
      }
    }
    if (!writes) continue;
    float y = f[c.eG(t)] * sum[t][0];
#pragma unroll
    for (int r = 0; r <= t; ++r) y = fmaf(f[c.mix(t, r)], f[c.u(r) + own], y);
    y = (y + f[c.skip(t) + own]) * f[c.gate(t) + own];
    const int64_t at = it.b * p.yb + t * p.ys + (int64_t)it.h * p.V + it.v + own;
    if (p.y_f32)
      static_cast<float *>(p.y)[at] = y;
    else
      static_cast<__nv_bfloat16 *>(p.y)[at] = __float2bfloat16_rn(y);
  }
}

// A warp whose wait ran out leaves: it touches no stage and arrives nowhere any more, so that the
// others' waits run out behind it and a state is the call's, or as it was.
template <typename S, int LPR, int PP, int TM>
__global__ void __launch_bounds__(SD_THREADS, sd_blocks(TM))
ssm_decode_ring_kernel(SsmDecodeParams p, int items) {
  extern __shared__ __align__(128) unsigned char ring[];
  __shared__ uint64_t full[SD_STAGES], ready[SD_STAGES], done[SD_STAGES], empty[SD_STAGES];
  constexpr int WARP_ROWS = SD_ROWS * 32 / LPR;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int role = warp < SD_WARPS ? 0 : warp < SD_WARPS + SD_PREP ? 1 : warp - SD_WARPS - SD_PREP + 2;
  const int coef_bytes = SdCoef(p.K, p.rows, p.T).bytes();
  if (tid == 0) {
    for (int s = 0; s < SD_STAGES; ++s) {
      ptx::mbar_init(&full[s], 1);
      ptx::mbar_init(&ready[s], 1);
      ptx::mbar_init(&done[s], SD_WARPS);
      ptx::mbar_init(&empty[s], 1);
    }
    ptx::fence_mbar_init();
  }
  __syncthreads();
  if (!bounds_ok(p.rows > 0 && p.rows <= SD_WARPS * WARP_ROWS &&
                     p.rows * p.K * (int)sizeof(S) <= (int)SD_TILE,
                 p.err))
    return;
  bool ok = true;
  auto wait = [&](uint64_t *bar, int use) {
    ok = ptx::mbar_wait_bounded(bar, (uint32_t)(use & 1), ok ? ptx::role_polls(role) : 1u) && ok;
  };
  auto item_at = [&](int i) {
    SdItem it;
    it.v = i % p.vblocks * p.rows;
    it.end = min(it.v + p.rows, p.V);
    const int bh = i / p.vblocks;
    it.b = bh / p.H;
    it.h = bh % p.H;
    it.slot = p.slots ? p.slots[it.b] : it.b;
    return it;
  };
  auto good = [&](const SdItem &it) { return it.slot >= 0 && it.slot < p.pool; };
  auto tile_of = [&](const SdItem &it) {
    return static_cast<S *>(p.state) + (((int64_t)it.slot * p.H + it.h) * p.V + it.v) * p.K;
  };
  auto bytes_of = [&](const SdItem &it) {
    return (uint32_t)((it.end - it.v) * p.K * (int)sizeof(S));
  };
  auto coef = [&](int s) {
    return reinterpret_cast<float *>(ring + SD_STAGES * SD_TILE + s * coef_bytes);
  };
  int n = 0;  // items of this block so far
  if (warp < SD_WARPS) {
    for (int i = blockIdx.x; i < items; i += gridDim.x, ++n) {
      const int s = n % SD_STAGES;
      const SdItem it = item_at(i);
      wait(&ready[s], n / SD_STAGES);
      wait(&full[s], n / SD_STAGES);
      if (!__all_sync(~0u, ok)) break;
      if (good(it)) {
        if (warp * WARP_ROWS < p.rows)
          ssm_decode_tile<S, LPR, PP, TM>(p, it, warp * WARP_ROWS,
                                          reinterpret_cast<S *>(ring + s * SD_TILE), coef(s));
      } else {
        if (tid == 0) record_error(p.err, GDN_ERR_BAD_SLOT);
        for (int t = 0; t < p.T; ++t)
          for (int r = it.v + tid; r < it.end; r += 32 * SD_WARPS) {
            const int64_t at = it.b * p.yb + t * p.ys + (int64_t)it.h * p.V + r;
            if (p.y_f32)
              static_cast<float *>(p.y)[at] = 0.f;
            else
              static_cast<__nv_bfloat16 *>(p.y)[at] = __float2bfloat16_rn(0.f);
          }
      }
      ptx::fence_proxy_async_smem();
      __syncwarp();
      if (lane == 0) ptx::mbar_arrive(&done[s]);
    }
  } else if (warp < SD_WARPS + SD_PREP) {
    for (int i = blockIdx.x; i < items; i += gridDim.x, ++n) {
      if (n % SD_PREP != warp - SD_WARPS) continue;
      const int s = n % SD_STAGES;
      const SdItem it = item_at(i);
      if (n >= SD_STAGES) wait(&done[s], n / SD_STAGES - 1);
      if (!__all_sync(~0u, ok)) break;
      ssm_decode_prepare<TM>(p, it, coef(s));
      __syncwarp();
      if (lane == 0) ptx::mbar_arrive(&ready[s]);
    }
  } else if (warp == SD_WARPS + SD_PREP) {
    for (int i = blockIdx.x; i < items; i += gridDim.x, ++n) {
      const int s = n % SD_STAGES;
      const SdItem it = item_at(i);
      if (n >= SD_STAGES) wait(&empty[s], n / SD_STAGES - 1);
      if (!__all_sync(~0u, ok)) break;
      if (lane == 0) {
        if (good(it)) {
          const uint32_t bytes = bytes_of(it);
          ptx::mbar_arrive_expect_tx(&full[s], bytes);
          ptx::bulk_g2s(ring + s * SD_TILE, tile_of(it), bytes, &full[s]);
        } else {
          ptx::mbar_arrive(&full[s]);
        }
      }
      __syncwarp();
    }
    // the last copies land before the warp ends, whoever else waits for them
    for (int k = max(0, n - SD_STAGES); k < n; ++k)
      ok = ptx::mbar_wait_bounded(&full[k % SD_STAGES], (uint32_t)(k / SD_STAGES & 1), 1u << 22) && ok;
  } else {
    for (int i = blockIdx.x; i < items; i += gridDim.x, ++n) {
      const int s = n % SD_STAGES;
      const SdItem it = item_at(i);
      wait(&done[s], n / SD_STAGES);
      if (!__all_sync(~0u, ok)) break;
      if (lane == 0) {
        if (good(it)) ptx::bulk_s2g(tile_of(it), ring + s * SD_TILE, bytes_of(it));
        ptx::bulk_commit();
        if (n > 0) {  // the store before has read its tile
          ptx::bulk_wait_read<1>();
          ptx::mbar_arrive(&empty[(n - 1) % SD_STAGES]);
        }
      }
      __syncwarp();
    }
    if (lane == 0) ptx::bulk_wait<0>();
  }
  if (!ok && lane == 0) record_error(p.err, GDN_ERR_TIMEOUT);
}

template <typename S, int LPR, int PP, int TM>
cudaError_t launch_decode(SsmDecodeParams &p, cudaStream_t stream) {
  constexpr int ROWS = SD_WARPS * SD_ROWS * 32 / LPR;
  const int64_t bh = (int64_t)p.B * p.H;
  // The ring pays once every block has an item (requests of 64 heads, bf16 states of
  // 64 x 128, ring / direct, us: 8 requests 6.2 / 6.3, 16 8.0 / 9.3, 64 20.3 / 28.9,
  // 256 93.1 / 152.5).
  const int blocks = sd_blocks(TM) * sm_count();
  const int rows = std::min(ROWS, (int)(SD_TILE / (p.K * sizeof(S))));
  const int vblocks = (p.V + rows - 1) / rows;
  if (bh * vblocks >= blocks && bh * vblocks <= 0x7fff0000) {
    p.vblocks = vblocks;
    p.rows = (p.V + vblocks - 1) / vblocks;
    const int smem = SD_STAGES * ((int)SD_TILE + SdCoef(p.K, p.rows, p.T).bytes());
    const cudaError_t e = cudaFuncSetAttribute(ssm_decode_ring_kernel<S, LPR, PP, TM>,
                                               cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
    if (e != cudaSuccess) return e;
    ssm_decode_ring_kernel<S, LPR, PP, TM>
        <<<blocks, SD_THREADS, smem, stream>>>(p, (int)(bh * vblocks));
  } else {
    p.vblocks = (p.V + ROWS - 1) / ROWS;
    ssm_decode_kernel<S, LPR, PP, TM>
        <<<(unsigned)(bh * p.vblocks), 32 * SD_WARPS, 0, stream>>>(p);
  }
  return cudaGetLastError();
}

template <typename S, int LPR, int PP>
cudaError_t launch_tokens(SsmDecodeParams &p, cudaStream_t stream) {
  if (p.T == 1) return launch_decode<S, LPR, PP, 1>(p, stream);
  if (p.T == 2) return launch_decode<S, LPR, PP, 2>(p, stream);
  return launch_decode<S, LPR, PP, 4>(p, stream);
}

template <typename S>
cudaError_t launch_pieces(SsmDecodeParams &p, cudaStream_t stream) {
  const int pieces = p.K * (int)sizeof(S) / 16;
  if (pieces <= 8) return launch_tokens<S, 8, 1>(p, stream);
  if (pieces <= 16) return launch_tokens<S, 16, 1>(p, stream);
  if (pieces <= 32) return launch_tokens<S, 32, 1>(p, stream);
  return launch_tokens<S, 32, 2>(p, stream);
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
  CHECK_THAT(a.T <= MAX_TOKENS, GDN_ERR_UNSUPPORTED, "T (%d) must be at most %d", a.T, MAX_TOKENS);
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

// Copies what both forms' parameters share.  A stride that no second token or batch row
// uses may be anything (a tensor map takes none of 2^40 bytes): dense rows instead, 0.
template <typename P, typename Args>
void set_tokens(P &p, const Args &a) {
  p.x = a.x; p.z = a.z; p.Bm = a.Bm; p.Cm = a.Cm; p.dt = a.dt;
  p.A_log = a.A_log; p.D = a.D; p.dt_bias = a.dt_bias; p.y = a.y;
  const bool many = a.B > 1, tokens = a.T > 1;
  const int64_t hv = (int64_t)a.H * a.V, gk = (int64_t)a.Hg * a.K;
  p.xs = tokens ? a.x_stride : hv; p.xb = many ? a.x_batch_stride : 0;
  p.zs = tokens ? a.z_stride : hv; p.zb = many ? a.z_batch_stride : 0;
  p.bs = tokens ? a.Bm_stride : gk; p.bb = many ? a.Bm_batch_stride : 0;
  p.cs = tokens ? a.Cm_stride : gk; p.cb = many ? a.Cm_batch_stride : 0;
  p.dts = tokens ? a.dt_stride : a.H; p.dtb = many ? a.dt_batch_stride : 0;
  p.ys = tokens ? a.y_stride : hv; p.yb = many ? a.y_batch_stride : 0;
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

// Segment length when the caller leaves it open: the one of least estimated time,
// in tokens that are walked one after another.  Whole sequences are walked in one
// pass.  Segments are walked in two, the first without y (together 1.4 times one on
// the tensor cores, 1.85 times on CUDA cores), and cost a second start and, for the
// later ones, the states of all segments before; on the tensor cores once for every
// block that an SM takes after another, on CUDA cores behind the three other blocks
// of the SM.  `held` blocks run at a time:
// sequences of one length take whole waves of them; packed ones, whose lengths the
// host does not know, queue, with half a block's walk left idle at the end (the
// longest is taken to be half as long again as the mean).
// One sequence of 4096 tokens (states of 64 x 128), whole / segments, us: bf16
// 8 heads 80 / 35, 32 heads 81 / 47, 64 heads 82 / 77, 80 heads 82 / 116;
// float32 8 heads 1019 / 115, 64 heads 1398 / 619, 120 heads 1470 / 1063.  Eight
// packed prompts (bf16), 32068 tokens and 32 heads 277 / 274 to 310, 12001 tokens
// and 16 heads 55 / 60 to 109.
int choose_segment(const SsmParams &p, bool tc) {
  const int cols = tc ? 64 : 32;  // of a block's state tile; one block an SM, or four
  const double chains = (double)p.H * ((p.V + cols - 1) / cols);
  const double held = (tc ? 1 : 4) * sm_count();
  const double passes = tc ? 1.4 : 1.85, start = tc ? 400 : 64, state = tc ? 50 : 8;
  const int64_t longest = p.cu ? std::min<int64_t>(p.T, (int64_t)p.T * 3 / (2 * p.N)) : p.T;
  auto walked = [&](int64_t seg, int64_t pieces) {
    return p.cu ? std::max<double>(seg, p.T * chains / held + seg / 2)
                : std::ceil(chains * p.N * pieces / held) * seg;
  };
  const int unit = tc ? SSM_UNIT : SSM_UNIT / 2;
  // (one unit holds it whole; no tokens, or a mean of less than one, too)
  if (longest <= unit) return SSM_WHOLE;
  int best = SSM_WHOLE;
  double least = walked(longest, 1) + start / 2;
  for (int n = 2; n <= 64; ++n) {
    const int64_t seg = ((longest + n - 1) / n + unit - 1) / unit * unit;
    const int64_t pieces = (longest + seg - 1) / seg;
    if (pieces < 2) break;
    const double tokens = walked(seg, pieces), starts = tc ? tokens / seg : 1;
    const double cost = passes * tokens + starts * (start + state * pieces);
    if (cost < least) {
      least = cost;
      best = (int)seg;
    }
  }
  return best;
}

// The kernels' parameters of a checked call, but for the workspace and the error word.
gdn_status_t chunk_params(const ssm_chunk_args &a, SsmParams &p) {
  set_tokens(p, a);
  p.N = a.N;
  p.h0 = a.h0; p.ht = a.ht; p.cu = a.cu_seqlens;
  p.seg = a.segment_tokens > 0 ? a.segment_tokens
                               : choose_segment(p, ssm_tc_supported(p, a.dtype == GDN_BF16));
  const int64_t longest = a.T;  // no sequence has more tokens
  const int64_t per = longest > p.seg ? (longest + p.seg - 1) / p.seg : 1;
  const int64_t items = a.cu_seqlens ? (a.N + (longest > p.seg ? longest / p.seg : 0)) : a.N * per;
  CHECK_THAT(items <= 0x7fffffff, GDN_ERR_UNSUPPORTED,
             "%lld segments of %d tokens are too many for one call", (long long)items, p.seg);
  p.items = (int)items;
  return GDN_OK;
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
  SsmParams p{};
  st = chunk_params(*a, p);
  if (st != GDN_OK) return st;
  *bytes = chunk_workspace(p);
  return GDN_OK;
}

gdn_status_t ssm_chunk_fwd(const ssm_chunk_args *a, gdn_stream_t stream) {
  (void)set_host_error(GDN_OK, "");
  CHECK_THAT(a != nullptr, GDN_ERR_INVALID_ARG, "args is NULL");
  gdn_status_t st = check_chunk_args(*a);
  if (st != GDN_OK) return st;
  SsmParams p{};
  st = chunk_params(*a, p);
  if (st != GDN_OK) return st;
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
  CHECK_THAT(a->V <= MAX_TOKENS, GDN_ERR_UNSUPPORTED, "V (%d) must be at most %d", a->V, MAX_TOKENS);
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
  p.state = a->state; p.slots = a->slot_indices; p.pool = a->pool; p.none = -0.f;
  const int wide = 16 / (int)dtype_bytes(a->dtype);
  p.whole_bc = aligned_to(a->Bm, 16) && aligned_to(a->Cm, 16) && p.bs % wide == 0 &&
               p.bb % wide == 0 && p.cs % wide == 0 && p.cb % wide == 0;
  p.err = device_error_word();
  if (p.err == nullptr) return launch_status(cudaGetLastError(), "device error word");
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  p.tok_f32 = a->dtype == GDN_F32;
  const cudaError_t e = a->state_dtype == GDN_BF16 ? launch_pieces<__nv_bfloat16>(p, s)
                                                   : launch_pieces<float>(p, s);
  return launch_status(e, "scan token launch");
}

}  // extern "C"
