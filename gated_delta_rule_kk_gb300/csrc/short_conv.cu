// Short causal depthwise convolution: over prompts, its gradient, and for
// single tokens against pooled states.
//
// Per channel, p_t = bias + sum_{i<W} w_i x_{t-W+1+i} and y = act(p), W <= 4:
// 2 W operations for one element read and one written, so every form is bound
// by memory.  A thread owns a few channels and walks a run of tokens with the
// last W - 1 rows in registers, so a row is read once but for the W - 1 rows
// beside each run.  Sums are float32.
//
// Long calls stream the rows through a ring of TMA tiles in shared memory
// (conv_ring_kernel): what is on its way is then bounded by shared memory, not
// by the registers, of which the gradient needs most for its sums.  Short calls,
// and rows that TMA cannot address, read them into registers.
//
// Measured (bf16, W = 4; share of the card's copy rate): two prompts of 4096 tokens
// and 6144 channels 40 us, 74%; eight packed prompts of 32068 tokens, 4352 channels
// 105 us, 78%; the gradient of the first 74 us, 60%; one token of 256 requests, 8192
// channels 7.8 us, 64%, of one request 2.4 us, a launch.  What the gradient is short of
// is warps: twelve of an SM compute, beside 192 KB that can be on its way.
#include <algorithm>
#include <initializer_list>
#include <type_traits>

#include "abi_check.h"
#include "gdn_common.cuh"
#include "ptx.cuh"
#include "rows.cuh"
#include "tensor_map.h"

namespace gdn {
namespace {

constexpr int CV_BATCH = 4;      // rows a thread has on the way at a time
constexpr int CV_MAX_THREADS = 256;
constexpr int CV_PIECE = 8;      // bytes of a bf16 row that a thread takes (16 of fp32)
constexpr int CV_BLOCKS = 2;     // blocks an SM holds at least (bounds the registers)
constexpr int CB_PIECE = 8, CB_BLOCKS = 1;  // the same of the gradient

// Weights of channels c .. c + VEC as w[tap][channel]: their VEC * W values are
// consecutive and, for VEC > 1, a multiple of 16 bytes at a 16-byte boundary.
template <int VEC, int W>
__device__ __forceinline__ void load_weights(float (&w)[W][VEC], float (&bias)[VEC],
                                             const void *weight, const void *b, bool f32, int c) {
  auto read = [&](auto tag) {
    using TW = decltype(tag);
    const TW *src = static_cast<const TW *>(weight) + (size_t)c * W;
    constexpr int PIECE = VEC == 1 ? 1 : 16 / (int)sizeof(TW);
    if constexpr (VEC * W % PIECE == 0) {
      float f[VEC * W];
#pragma unroll
      for (int i = 0; i < VEC * W; i += PIECE) {
        Row<TW, PIECE> r;
        r.load(src + i);
        r.widen(f + i);
      }
#pragma unroll
      for (int i = 0; i < VEC * W; ++i) w[i % W][i / W] = f[i];
    } else {
#pragma unroll
      for (int i = 0; i < VEC * W; ++i) w[i % W][i / W] = to_f32(src[i]);
    }
#pragma unroll
    for (int e = 0; e < VEC; ++e) bias[e] = b ? to_f32(static_cast<const TW *>(b)[c + e]) : 0.f;
  };
  if (f32)
    read(0.f);
  else
    read(__nv_bfloat16());
}

struct ConvSeqs {
  const int32_t *cu;
  int B, T, N;
};

// The sequence that token t of batch row b belongs to: the last one that does
// not start after it (0 <= t < T, offsets checked).
__device__ __forceinline__ int conv_sequence_of(const ConvSeqs &q, int b, int t) {
  if (q.cu == nullptr) return b;
  int lo = 0, hi = q.N;  // cu[lo] <= t < cu[hi]
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (q.cu[mid] <= t)
      lo = mid;
    else
      hi = mid;
  }
  return lo;
}

struct ConvParams {
  const void *x, *weight, *bias, *h0;
  void *ht, *y;
  int *err;
  ConvSeqs q;
  int64_t xs, xb, ys, yb;
  int D, silu, w_f32;
  int run, tiles;  // tokens of a run, runs of a batch row
};

// The rows before token t of a sequence that starts at bos: x's own, or the
// state's (zeros without one).  `xr` is the sequence's batch row.
template <typename T, int VEC, int W>
__device__ __forceinline__ void load_before(float (*win)[VEC], const T *xr, int64_t xs,
                                            const T *state, int D, int bos, int t) {
#pragma unroll
  for (int j = 0; j < W - 1; ++j) {
    const int pos = t - (W - 1) + j - bos;
    Row<T, VEC> r;
    if (pos >= 0)
      r.load(xr + (int64_t)(bos + pos) * xs);
    else if (state)
      r.load(state + (int64_t)(pos + W - 1) * D);
    else
      r.zero();
    r.widen(win[j]);
  }
}

// grid: x = runs of every batch row, then (with ht) one block per sequence;
// y = channel blocks.
template <typename T, int VEC, int W>
__global__ void __launch_bounds__(CV_MAX_THREADS, CV_BLOCKS) conv_fwd_kernel(ConvParams p) {
  if (!offsets_ok(p.q.cu, p.q.N, p.q.T, p.err)) return;
  const int c = (blockIdx.y * blockDim.x + threadIdx.x) * VEC;
  if (c >= p.D) return;
  const int runs = p.q.B * p.tiles;
  const T *x = static_cast<const T *>(p.x) + c;
  const T *h0 = p.h0 ? static_cast<const T *>(p.h0) + c : nullptr;
  if ((int)blockIdx.x >= runs) {
    // the last W - 1 rows of sequence n
    const int n = blockIdx.x - runs;
    const int bos = p.q.cu ? p.q.cu[n] : 0, eos = p.q.cu ? p.q.cu[n + 1] : p.q.T;
    if (!bounds_ok(n < p.q.N && bos >= 0 && bos <= eos && eos <= p.q.T, p.err)) return;
    const T *xr = x + (p.q.cu ? 0 : n) * p.xb;
    T *ht = static_cast<T *>(p.ht) + (int64_t)n * (W - 1) * p.D + c;
    for (int j = 0; j < W - 1; ++j) {
      const int pos = eos - bos - (W - 1) + j;
      Row<T, VEC> r;
      if (pos >= 0)
        r.load(xr + (int64_t)(bos + pos) * p.xs);
      else if (h0)
        r.load(h0 + ((int64_t)n * (W - 1) + pos + W - 1) * p.D);
      else
        r.zero();
      r.store(ht + (int64_t)j * p.D);
    }
    return;
  }
  const int b = blockIdx.x / p.tiles;
  int t = (blockIdx.x % p.tiles) * p.run;
  const int t1 = t + min(p.run, p.q.T - t);
  if (!bounds_ok(b < p.q.B && t < t1, p.err)) return;
  const T *xr = x + b * p.xb;
  T *yr = static_cast<T *>(p.y) + b * p.yb + c;
  float w[W][VEC], bias[VEC];
  load_weights<VEC, W>(w, bias, p.weight, p.bias, p.w_f32, c);
  for (int n = conv_sequence_of(p.q, b, t); t < t1; ++n) {
    const int bos = p.q.cu ? p.q.cu[n] : 0, end = min(t1, p.q.cu ? p.q.cu[n + 1] : p.q.T);
    if (t >= end) continue;  // an empty sequence
    Row<T, VEC> next[CV_BATCH];
    auto fetch = [&](int at) {
#pragma unroll
      for (int k = 0; k < CV_BATCH; ++k)
        if (at + k < end) next[k].load(xr + (int64_t)(at + k) * p.xs);
    };
    fetch(t);
    float f[W - 1 + CV_BATCH][VEC];
    load_before<T, VEC, W>(f, xr, p.xs, h0 ? h0 + (int64_t)n * (W - 1) * p.D : nullptr, p.D, bos, t);
    for (; t < end; t += CV_BATCH) {
#pragma unroll
      for (int k = 0; k < CV_BATCH; ++k) next[k].widen(f[W - 1 + k]);
      fetch(t + CV_BATCH);
#pragma unroll
      for (int k = 0; k < CV_BATCH; ++k) {
        if (t + k >= end) break;
        float acc[VEC];
#pragma unroll
        for (int e = 0; e < VEC; ++e) acc[e] = bias[e];
#pragma unroll
        for (int i = 0; i < W; ++i) fma_row<VEC>(acc, w[i], f[k + i]);
        if (p.silu) {
#pragma unroll
          for (int e = 0; e < VEC; ++e) acc[e] = silu(acc[e]);
        }
        Row<T, VEC> out;
        out.round(acc);
        out.store(yr + (int64_t)(t + k) * p.ys);
      }
#pragma unroll
      for (int j = 0; j < W - 1; ++j)
#pragma unroll
        for (int e = 0; e < VEC; ++e) f[j][e] = f[CV_BATCH + j][e];
    }
    t = end;
  }
}

// ---------------------------------------------------------------- gradient

constexpr int CB_RUNS = 8;  // runs (warps) of a block

struct ConvBwdParams {
  const void *dy, *x, *weight, *bias, *h0, *dht;
  void *dx, *dh0;
  float *part;  // [blocks along time][W + 1][D], or NULL
  int *err;
  ConvSeqs q;
  int64_t gs, gb, xs, xb, ds, db;
  int D, silu, w_f32;
  int run, tiles;  // tokens of a warp's run, blocks (of CB_RUNS runs) of a batch row
};

// Warp y of a block walks one run [lo, hi) of tokens for 32 * VEC channels.
// dx_t = sum_i w_i dp_{t+W-1-i} needs dp of the W - 1 tokens after t, so the
// walk goes W - 1 tokens past the run's (or the sequence's) end, where dp past
// the sequence is zero, and row u - (W - 1) is written as token u is taken.
// The run that holds a sequence's first token writes its dh0.  dweight and
// dbias sums of the run's own tokens stay in registers, are added over the
// block's runs in shared memory and leave as one partial sum per block.
template <typename T, int VEC, int W>
__global__ void __launch_bounds__(32 * CB_RUNS, CB_BLOCKS) conv_bwd_kernel(ConvBwdParams p) {
  __shared__ float red[CB_RUNS][32 * VEC + 4];
  if (!offsets_ok(p.q.cu, p.q.N, p.q.T, p.err)) return;
  const int lane = threadIdx.x;
  const int c = (blockIdx.y * 32 + lane) * VEC;
  const bool live = c < p.D;
  const int blocks = p.q.B * p.tiles;
  if ((int)blockIdx.x >= blocks) {
    // a sequence without tokens: its final state is its initial state
    const int n = blockIdx.x - blocks;
    if (!bounds_ok(n < p.q.N, p.err)) return;
    const int len = p.q.cu ? p.q.cu[n + 1] - p.q.cu[n] : p.q.T;
    if (len > 0 || !live || threadIdx.y) return;
    for (int j = 0; j < W - 1; ++j) {
      const int64_t at = ((int64_t)n * (W - 1) + j) * p.D + c;
      Row<T, VEC> r;
      if (p.dht)
        r.load(static_cast<const T *>(p.dht) + at);
      else
        r.zero();
      r.store(static_cast<T *>(p.dh0) + at);
    }
    return;
  }
  float w[W][VEC], bias[VEC], dw[W][VEC], db[VEC];
#pragma unroll
  for (int e = 0; e < VEC; ++e) {
    db[e] = 0.f;
#pragma unroll
    for (int i = 0; i < W; ++i) dw[i][e] = 0.f;
  }
  const int b = blockIdx.x / p.tiles;
  if (!bounds_ok(b < p.q.B, p.err)) return;
  // (a block's last runs may lie past the end: their products pass 31 bits)
  const int64_t warp_run = (int64_t)(blockIdx.x % p.tiles) * CB_RUNS + threadIdx.y;
  const int lo = (int)min((int64_t)p.q.T, warp_run * p.run);
  const int hi = lo + min(p.run, p.q.T - lo);
  if (live && lo < hi) {
    load_weights<VEC, W>(w, bias, p.weight, p.bias, p.w_f32, c);
    const T *xr = static_cast<const T *>(p.x) + b * p.xb + c;
    const T *gr = static_cast<const T *>(p.dy) + b * p.gb + c;
    T *dxr = static_cast<T *>(p.dx) + b * p.db + c;
    int t0 = lo;
    for (int n = conv_sequence_of(p.q, b, lo); t0 < hi; ++n) {
      const int bos = p.q.cu ? p.q.cu[n] : 0, eos = p.q.cu ? p.q.cu[n + 1] : p.q.T;
      if (t0 >= eos) continue;  // an empty sequence
      const int own = min(eos, hi), last = min(eos, hi + W - 1);
      const int64_t st = (int64_t)n * (W - 1) * p.D + c;
      Row<T, VEC> nx[CV_BATCH], ng[CV_BATCH];
      auto fetch = [&](int at) {
#pragma unroll
        for (int k = 0; k < CV_BATCH; ++k)
          if (at + k < last) {
            nx[k].load(xr + (int64_t)(at + k) * p.xs);
            ng[k].load(gr + (int64_t)(at + k) * p.gs);
          }
      };
      fetch(t0);
      float f[W - 1 + CV_BATCH][VEC], d[W - 1 + CV_BATCH][VEC];
      load_before<T, VEC, W>(f, xr, p.xs, p.h0 ? static_cast<const T *>(p.h0) + st : nullptr, p.D,
                             bos, t0);
#pragma unroll
      for (int j = 0; j < W - 1; ++j)
#pragma unroll
        for (int e = 0; e < VEC; ++e) d[j][e] = 0.f;
      for (int u = t0; u < own + W - 1; u += CV_BATCH) {
#pragma unroll
        for (int k = 0; k < CV_BATCH; ++k) {
          nx[k].widen(f[W - 1 + k]);
          ng[k].widen(d[W - 1 + k]);
        }
        fetch(u + CV_BATCH);
#pragma unroll
        for (int k = 0; k < CV_BATCH; ++k) {
          float *dp = d[W - 1 + k];
          if (u + k < last) {
            if (p.silu) {
              float acc[VEC];
#pragma unroll
              for (int e = 0; e < VEC; ++e) acc[e] = bias[e];
#pragma unroll
              for (int i = 0; i < W; ++i) fma_row<VEC>(acc, w[i], f[k + i]);
#pragma unroll
              for (int e = 0; e < VEC; ++e) {
                // silu'(p) = s (1 + p (1 - s)), s = 1 / (1 + e^-p)
                const float s = __fdividef(1.f, 1.f + __expf(-acc[e]));
                dp[e] *= s * fmaf(acc[e], 1.f - s, 1.f);
              }
            }
            if (u + k < own) {
#pragma unroll
              for (int i = 0; i < W; ++i) fma_row<VEC>(dw[i], dp, f[k + i]);
#pragma unroll
              for (int e = 0; e < VEC; ++e) db[e] += dp[e];
            }
          } else {
#pragma unroll
            for (int e = 0; e < VEC; ++e) dp[e] = 0.f;
          }
          const int t = u + k - (W - 1);
          const bool token = t >= t0 && t < own, state = t < bos && t0 == bos && p.dh0 != nullptr;
          if (!token && !state) continue;
          float acc[VEC];
          const int back = t - eos + W - 1;  // the row of dht that row t became
          if (p.dht && back >= 0) {
            Row<T, VEC> r;
            r.load(static_cast<const T *>(p.dht) + st + (int64_t)back * p.D);
            r.widen(acc);
          } else {
#pragma unroll
            for (int e = 0; e < VEC; ++e) acc[e] = 0.f;
          }
#pragma unroll
          for (int i = 0; i < W; ++i) fma_row<VEC>(acc, w[i], d[W - 1 + k - i]);
          Row<T, VEC> out;
          out.round(acc);
          if (token)
            out.store(dxr + (int64_t)t * p.ds);
          else
            out.store(static_cast<T *>(p.dh0) + st + (int64_t)(t - bos + W - 1) * p.D);
        }
#pragma unroll
        for (int j = 0; j < W - 1; ++j)
#pragma unroll
          for (int e = 0; e < VEC; ++e) {
            f[j][e] = f[CV_BATCH + j][e];
            d[j][e] = d[CV_BATCH + j][e];
          }
      }
      t0 = own;
    }
  }
  if (p.part == nullptr) return;
  float *part = p.part + (int64_t)blockIdx.x * (W + 1) * p.D;
#pragma unroll
  for (int i = 0; i <= W; ++i) {
    __syncthreads();
#pragma unroll
    for (int e = 0; e < VEC; ++e) red[threadIdx.y][lane * VEC + e] = i < W ? dw[i < W ? i : 0][e] : db[e];
    __syncthreads();
    for (int e = threadIdx.y * 32 + lane; e < 32 * VEC; e += 32 * CB_RUNS) {
      const int ch = blockIdx.y * 32 * VEC + e;
      if (ch >= p.D) continue;
      float s = 0.f;
#pragma unroll
      for (int r = 0; r < CB_RUNS; ++r) s += red[r][e];
      part[(int64_t)i * p.D + ch] = s;
    }
  }
}

// dweight and dbias from the blocks' partial sums: block (32 channels, one tap
// or the bias), warp y adds every 8th partial sum, then the warps in order.
template <int W>
__global__ void __launch_bounds__(256) conv_bwd_sum_kernel(const float *part, int blocks, int D,
                                                           float *dweight, float *dbias, ConvSeqs q,
                                                           int *err) {
  __shared__ float red[8][32];
  if (!offsets_ok(q.cu, q.N, q.T, err)) return;
  const int c = blockIdx.x * 32 + threadIdx.x, i = blockIdx.y;
  float s = 0.f;
  if (c < D) {
#pragma unroll 4
    for (int k = threadIdx.y; k < blocks; k += 8) s += part[((int64_t)k * (W + 1) + i) * D + c];
  }
  red[threadIdx.y][threadIdx.x] = s;
  __syncthreads();
  if (threadIdx.y != 0 || c >= D) return;
#pragma unroll
  for (int k = 1; k < 8; ++k) s += red[k][threadIdx.x];
  if (i < W) {
    if (dweight) dweight[(int64_t)c * W + i] = s;
  } else if (dbias) {
    dbias[c] = s;
  }
}

// ---------------------------------------------------------------- the ring

// A block owns a range of channels (two TMA boxes of bf16 rows, one of float32)
// and walks a run of tokens, whose rows another warp loads 8 at a time.
constexpr int CR_BOX = 256;   // channels of a TMA box
constexpr int CR_STAGE = 8;   // rows of a stage
constexpr int CR_LEAST = 16;  // tokens of a run, below which a call is short
template <typename T, bool BWD>
struct ConvRing {
  static constexpr int BOXES = sizeof(T) == 2 ? 2 : 1, CHANNELS = BOXES * CR_BOX;
  static constexpr int VEC = 8 / (int)sizeof(T), THREADS = CHANNELS / VEC;
  static constexpr int ROW = CR_BOX * (int)sizeof(T);  // bytes of a box's row
  static constexpr int BOX = CR_STAGE * ROW;
  static constexpr int STAGE = BOXES * BOX * (BWD ? 2 : 1);
  // Stages, and blocks that an SM holds: three of the gradient's take 192 of 227 KB and
  // 128 registers a thread for its sums and windows; either alone keeps a fourth out.
  static constexpr int STAGES = 4;
  static constexpr int BLOCKS = BWD ? 3 : 5;
};

struct ConvRingParams {
  const void *weight, *bias, *h0, *dht;
  void *out, *ht;  // y, ht or dx, dh0
  float *part;     // [B * runs][W + 1][D], or NULL
  int *err;
  ConvSeqs q;
  int64_t xs, xb, os, ob;
  const void *x;
  int D, silu, w_f32;
  int run, runs;  // tokens of a run, runs of a batch row
};

// The rows of a run are taken one after another, u = lo, lo + 1, ..; row u lives in
// slot u - lo mod 4 of a thread's registers.  Forward: y_u.  Gradient: dp_u from
// p_u, then dx of row u - (W - 1), whose last term dp_u is; the walk goes W - 1
// rows past the run, or ends with the sequence by taking dp as zero there.
template <typename T, int W, bool BWD>
__global__ void __launch_bounds__(ConvRing<T, BWD>::THREADS + 32, ConvRing<T, BWD>::BLOCKS)
conv_ring_kernel(const __grid_constant__ CUtensorMap tm_x,
                 const __grid_constant__ CUtensorMap tm_g, ConvRingParams p) {
  extern __shared__ __align__(128) unsigned char ring[];
  using R = ConvRing<T, BWD>;
  constexpr int VEC = R::VEC, S = R::STAGES;
  __shared__ uint64_t full[S], empty[S];
  const int tid = threadIdx.x, lane = tid & 31;
  if (!offsets_ok(p.q.cu, p.q.N, p.q.T, p.err)) return;
  const int runs = p.q.B * p.runs, c0 = blockIdx.y * R::CHANNELS, c = c0 + tid * VEC;
  if ((int)blockIdx.x >= runs) {
    // forward: the last W - 1 rows of sequence n; gradient: a sequence without
    // tokens, whose final state is its initial state
    const int n = blockIdx.x - runs;
    if (!bounds_ok(n < p.q.N, p.err)) return;
    if (tid >= R::THREADS || c >= p.D) return;
    const int bos = p.q.cu ? p.q.cu[n] : 0, eos = p.q.cu ? p.q.cu[n + 1] : p.q.T;
    if (BWD && eos > bos) return;
    const T *xr = static_cast<const T *>(p.x) + (p.q.cu ? 0 : n) * p.xb + c;
    const T *before = static_cast<const T *>(BWD ? p.dht : p.h0);
    T *to = static_cast<T *>(p.ht) + (int64_t)n * (W - 1) * p.D + c;
    for (int j = 0; j < W - 1; ++j) {
      const int pos = eos - bos - (W - 1) + j;
      Row<T, VEC> r;
      if (pos >= 0)
        r.load(xr + (int64_t)(bos + pos) * p.xs);
      else if (before)
        r.load(before + ((int64_t)n * (W - 1) + pos + W - 1) * p.D + c);
      else
        r.zero();
      r.store(to + (int64_t)j * p.D);
    }
    return;
  }
  const int b = blockIdx.x / p.runs, lo = blockIdx.x % p.runs * p.run;
  const int hi = lo + min(p.run, p.q.T - lo), stop = BWD ? min(p.q.T, hi + W - 1) : hi;
  if (!bounds_ok(b < p.q.B && lo < hi && c0 < p.D, p.err)) return;
  if (tid == 0) {
    for (int s = 0; s < S; ++s) {
      ptx::mbar_init(&full[s], 1);
      ptx::mbar_init(&empty[s], R::THREADS / 32);
    }
    ptx::fence_mbar_init();
  }
  __syncthreads();
  bool ok = true;
  auto wait = [&](uint64_t *bar, int use) {
    const int role = tid < R::THREADS ? 0 : 2;  // taking rows, loading
    ok = ptx::mbar_wait_bounded(bar, (uint32_t)(use & 1), ok ? ptx::role_polls(role) : 1u) && ok;
  };
  if (tid >= R::THREADS) {
    const int boxes = p.D - c0 > CR_BOX ? R::BOXES : 1;
    int m = 0;  // stages asked for
    for (int u = lo; u < stop; u += CR_STAGE, ++m) {
      const int s = m % S;
      if (m >= S) wait(&empty[s], m / S - 1);
      if (!__all_sync(~0u, ok)) break;
      if (lane == 0) ptx::mbar_arrive_expect_tx(&full[s], boxes * R::BOX * (BWD ? 2 : 1));
      __syncwarp();
      // one copy a lane: the copies of one thread complete one after another
      const int box = lane & 1, g = lane >> 1;
      if (box < boxes && g < (BWD ? 2 : 1))
        ptx::tma_load_3d(ring + s * R::STAGE + (g * R::BOXES + box) * R::BOX,
                         g ? (const void *)&tm_g : (const void *)&tm_x, c0 + box * CR_BOX, u, b,
                         &full[s]);
    }
    // the last copies land before the warp ends, whoever else waits for them
    for (int k = max(0, m - S); k < m; ++k)
      ok = ptx::mbar_wait_bounded(&full[k % S], (uint32_t)(k / S & 1), 1u << 22) && ok;
    if (!ok && lane == 0) record_error(p.err, GDN_ERR_TIMEOUT);
    return;
  }

  const bool live = c < p.D;
  float w[W][VEC], bias[VEC], f[4][VEC], d[4][VEC], dw[W][VEC], db[VEC];
  if (live) {
    load_weights<VEC, W>(w, bias, p.weight, p.bias, p.w_f32, c);
  } else {
#pragma unroll
    for (int e = 0; e < VEC; ++e) {
      bias[e] = 0.f;
#pragma unroll
      for (int i = 0; i < W; ++i) w[i][e] = 0.f;
    }
  }
#pragma unroll
  for (int e = 0; e < VEC; ++e) {
    db[e] = 0.f;
#pragma unroll
    for (int i = 0; i < W; ++i) dw[i][e] = 0.f;
#pragma unroll
    for (int i = 0; i < 4; ++i) f[i][e] = d[i][e] = 0.f;
  }
  const T *xr = static_cast<const T *>(p.x) + b * p.xb + c;
  T *outr = static_cast<T *>(p.out) + b * p.ob + c;
  // this thread's channels in the rows of a stage
  const unsigned char *mine = ring + tid * VEC / CR_BOX * R::BOX + tid * VEC % CR_BOX * sizeof(T);
  int n = conv_sequence_of(p.q, b, lo), bos = p.q.cu ? p.q.cu[n] : 0;
  int eos = p.q.cu ? p.q.cu[n + 1] : p.q.T, t0 = lo;
  int64_t st = 0;  // the sequence's rows of the states

  // Writes row t of dx, or of dh0 before the sequence, from the sum `acc`.
  auto emit = [&](int t, float *acc) {
    const bool token = t >= t0 && t < hi, state = t < bos && t0 == bos && p.ht != nullptr;
    if (!live || !(token || state)) return;
    const int back = t - eos + W - 1;  // the row of dht that row t became
    if (p.dht && back >= 0) {
      Row<T, VEC> r;
      float g[VEC];
      r.load(static_cast<const T *>(p.dht) + st + (int64_t)back * p.D);
      r.widen(g);
      add_row<VEC>(acc, acc, g);
    }
    Row<T, VEC> r;
    r.round(acc);
    r.store(token ? outr + (int64_t)t * p.os
                  : static_cast<T *>(p.ht) + st + (int64_t)(t - bos + W - 1) * p.D);
  };
  // The sequence ends before row u (slot k): the rows whose sums wait for it.
  auto flush = [&](int u, int k) {
#pragma unroll
    for (int m = W - 1; m >= 1; --m) {
      float acc[VEC];
#pragma unroll
      for (int e = 0; e < VEC; ++e) acc[e] = 0.f;
#pragma unroll
      for (int i = W - m; i < W; ++i) fma_row<VEC>(acc, w[i], d[(k - (m - W + 1 + i)) & 3]);
      emit(u - m, acc);
    }
  };
  // Row u belongs to sequence n: the rows before it.
  auto begin = [&](int u, int k) {
    t0 = u;
    st = (int64_t)n * (W - 1) * p.D + c;
    float win[W - 1][VEC];
#pragma unroll
    for (int j = 0; j < W - 1; ++j)
#pragma unroll
      for (int e = 0; e < VEC; ++e) win[j][e] = 0.f;
    if (live)
      load_before<T, VEC, W>(win, xr, p.xs, p.h0 ? static_cast<const T *>(p.h0) + st : nullptr, p.D,
                             bos, u);
#pragma unroll
    for (int j = 0; j < W - 1; ++j)
#pragma unroll
      for (int e = 0; e < VEC; ++e) {
        f[(k - (W - 1) + j) & 3][e] = win[j][e];
        d[(k - (W - 1) + j) & 3][e] = 0.f;
      }
  };
  auto next = [&](int u) {  // the sequence of row u, after the present one
    do {
      ++n;
      bos = eos;
      eos = p.q.cu[n + 1];
    } while (eos <= u);
  };
  begin(lo, 0);
  bool open = true;  // a sequence is being walked
  // Four rows from u0 on.  WITHIN: no sequence ends between them, so that they
  // are one run of arithmetic without branches (rows past `stop` are taken and
  // not kept).
  auto rows4 = [&](int u0, const unsigned char *rows, auto within) {
    constexpr bool WITHIN = decltype(within)::value;
    T *to = outr + (int64_t)(u0 - (BWD ? W - 1 : 0)) * p.os;
    Row<T, VEC> xs4[4], gs4[4];
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      xs4[k].load(reinterpret_cast<const T *>(rows + k * R::ROW));
      if (BWD) gs4[k].load(reinterpret_cast<const T *>(rows + R::BOXES * R::BOX + k * R::ROW));
    }
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      const int u = u0 + k;
      if (!WITHIN) {
        if (u >= stop || !open) break;
        if (u == eos) {
          if (BWD) flush(u, k);
          if (u >= hi) {
            open = false;
            break;
          }
          next(u);
          begin(u, k);
        }
      }
      xs4[k].widen(f[k]);
      float acc[VEC];
      if (!BWD || p.silu) {
        fma_rows<VEC>(acc, w[0], f[(k - (W - 1)) & 3], bias);
#pragma unroll
        for (int i = 1; i < W; ++i) fma_row<VEC>(acc, w[i], f[(k - (W - 1) + i) & 3]);
      }
      if (!BWD) {
        if (p.silu) silu_row<VEC>(acc, acc);
        Row<T, VEC> out;
        out.round(acc);
        if (live && u < hi) out.store(to + k * p.os);
        continue;
      }
      float *dp = d[k];
      gs4[k].widen(dp);
      if (p.silu) {
        // silu'(p) = s + s p (1 - s), s = 1 / (1 + e^-p)
        float sg[VEC], sp[VEC];
        sigmoid_row<VEC>(sg, acc);
        mul_row<VEC>(sp, sg, acc);
        mul_row<VEC>(acc, sg, sp);
        sub_row<VEC>(sp, sp, acc);
        add_row<VEC>(sp, sp, sg);
        mul_row<VEC>(dp, dp, sp);
      }
      if (WITHIN ? u0 < hi : u < hi) {
#pragma unroll
        for (int i = 0; i < W; ++i) fma_row<VEC>(dw[i], dp, f[(k - (W - 1) + i) & 3]);
        add_row<VEC>(db, db, dp);
      }
      mul_row<VEC>(acc, w[0], dp);
#pragma unroll
      for (int i = 1; i < W; ++i) fma_row<VEC>(acc, w[i], d[(k - i) & 3]);
      const int t = u - (W - 1);
      if (!WITHIN) {
        emit(t, acc);
      } else if (live && t >= t0 && t < hi) {
        Row<T, VEC> out;
        out.round(acc);
        out.store(to + k * p.os);
      }
    }
  };
  // (every stage is waited for, also past the end: none is left on its way; behind a wait that
  // ran out a warp arrives nowhere any more, so that no stage is asked for before its copy has
  // landed)
#pragma unroll 1
  for (int u0 = lo, r = 0; u0 < stop; u0 += 4, r += 4) {
    const int s = r / CR_STAGE % S;
    if (r % CR_STAGE == 0) wait(&full[s], r / CR_STAGE / S);
    const unsigned char *rows = mine + s * R::STAGE + r % CR_STAGE * R::ROW;
    // (the other form's: a sequence that ends in these rows or with the walk, rows
    // before a sequence's first token, and the sums of a part of four rows)
    if (open && eos > u0 && (eos >= u0 + 4 || (BWD ? eos > stop : eos >= stop)) &&
        (!BWD || ((t0 > bos || u0 - (W - 1) >= t0) && (u0 >= hi || u0 + 4 <= hi))))
      rows4(u0, rows, std::true_type());
    else if (open)
      rows4(u0, rows, std::false_type());
    if ((r + 4) % CR_STAGE == 0) {
      __syncwarp();
      if (lane == 0 && ok) ptx::mbar_arrive(&empty[s]);
    }
  }
  if (BWD && open && eos == stop) {  // the slot that row `stop` would have had
    const int k = (stop - lo) & 3;
    if (k == 0) flush(stop, 0);
    if (k == 1) flush(stop, 1);
    if (k == 2) flush(stop, 2);
    if (k == 3) flush(stop, 3);
  }
  if (BWD && p.part && live) {
    float *part = p.part + (int64_t)blockIdx.x * (W + 1) * p.D + c;
#pragma unroll
    for (int i = 0; i <= W; ++i) {
      const float *v = i < W ? dw[i < W ? i : 0] : db;
#pragma unroll
      for (int e = 0; e < VEC; e += 2)
        *reinterpret_cast<float2 *>(part + (int64_t)i * p.D + e) = make_float2(v[e], v[e + 1]);
    }
  }
  if (!ok && lane == 0) record_error(p.err, GDN_ERR_TIMEOUT);
}

// ---------------------------------------------------------------- single tokens

struct ConvDecodeParams {
  const void *x, *weight, *bias;
  void *state, *y;
  const int32_t *slots;
  int *err;
  int64_t xs, xb, ys, yb;
  int B, T, D, pool, silu, w_f32;
};

// grid: x = batch entries, y = channel blocks.  Everything a thread needs is
// asked for before anything is used: the call is a few microseconds long and
// bound by that one trip to memory.
template <typename T, int VEC, int W>
__global__ void __launch_bounds__(CV_MAX_THREADS) conv_decode_kernel(ConvDecodeParams p) {
  constexpr int TM = 4;
  const int c = (blockIdx.y * blockDim.x + threadIdx.x) * VEC;
  if (c >= p.D) return;
  const int b = blockIdx.x;
  if (!bounds_ok(b < p.B, p.err)) return;
  const T *x = static_cast<const T *>(p.x) + b * p.xb + c;
  T *y = static_cast<T *>(p.y) + b * p.yb + c;
  const int slot = p.slots ? p.slots[b] : b;
  Row<T, VEC> rows[W - 1 + TM];
#pragma unroll
  for (int t = 0; t < TM; ++t)
    if (t < p.T) rows[W - 1 + t].load(x + t * p.xs);
  float w[W][VEC], bias[VEC];
  load_weights<VEC, W>(w, bias, p.weight, p.bias, p.w_f32, c);
  if (slot < 0 || slot >= p.pool) {
    if (threadIdx.x == 0) record_error(p.err, GDN_ERR_BAD_SLOT);
    Row<T, VEC> r;
    r.zero();
    for (int t = 0; t < p.T; ++t) r.store(y + t * p.ys);
    return;
  }
  T *state = static_cast<T *>(p.state) + (int64_t)slot * (W - 1) * p.D + c;
#pragma unroll
  for (int j = 0; j < W - 1; ++j) rows[j].load(state + (int64_t)j * p.D);
#pragma unroll
  for (int t = 0; t < TM; ++t) {
    if (t >= p.T) break;
    float acc[VEC], f[VEC];
#pragma unroll
    for (int e = 0; e < VEC; ++e) acc[e] = bias[e];
#pragma unroll
    for (int i = 0; i < W; ++i) {
      rows[t + i].widen(f);
      fma_row<VEC>(acc, w[i], f);
    }
    if (p.silu) {
#pragma unroll
      for (int e = 0; e < VEC; ++e) acc[e] = silu(acc[e]);
    }
    Row<T, VEC> out;
    out.round(acc);
    out.store(y + t * p.ys);
  }
#pragma unroll
  for (int t = 1; t <= TM; ++t) {
    if (t != p.T) continue;
#pragma unroll
    for (int j = 0; j < W - 1; ++j) rows[t + j].store(state + (int64_t)j * p.D);
  }
}

// ---------------------------------------------------------------- host

// Threads of a block (a multiple of 32) that spread `pieces` evenly over the
// fewest blocks of at most 256.
int even_block(int64_t pieces) {
  const int64_t blocks = (pieces + CV_MAX_THREADS - 1) / CV_MAX_THREADS;
  const int64_t each = (pieces + blocks - 1) / blocks;
  return (int)((each + 31) / 32 * 32);
}

// Whether the rows of tensors with these addresses and strides can be taken in
// pieces of `vec` elements, each on a boundary of its size.
bool whole_pieces(int64_t D, int vec, int32_t dtype, std::initializer_list<const void *> tensors,
                  std::initializer_list<int64_t> strides) {
  if (D % vec != 0) return false;
  for (const void *t : tensors)
    if (!aligned_to(t, vec * dtype_bytes(dtype))) return false;
  for (int64_t s : strides)
    if (s % vec != 0) return false;
  return true;
}

// Tokens of a run: as few as let the whole call be on the GPU at once (with
// `threads` resident threads on an SM), so that no second wave is left
// half-empty.  A run reads W - 1 rows twice, from L2.  At least a batch, also of no
// tokens: runs are divided by.
int run_tokens(int64_t tokens, int64_t pieces, int threads) {
  const int64_t resident = (int64_t)sm_count() * threads;
  const int64_t run = std::max<int64_t>(1, (tokens * pieces + resident - 1) / resident);
  return (int)((run + CV_BATCH - 1) / CV_BATCH * CV_BATCH);
}

// Calls `f` with the element type and tap count as compile-time values.
template <typename F>
cudaError_t with_types(int32_t dtype, int W, F &&f) {
  auto taps = [&](auto t) {
    using T = decltype(t);
    if (W == 2) return f(T(), std::integral_constant<int, 2>());
    if (W == 3) return f(T(), std::integral_constant<int, 3>());
    return f(T(), std::integral_constant<int, 4>());
  };
  return dtype == GDN_BF16 ? taps(__nv_bfloat16()) : taps(0.f);
}

// [batch][token][channel], boxes of CR_BOX channels and a stage's tokens.
bool conv_map(CUtensorMap *m, const void *base, int elt, const ConvSeqs &q, int D, int64_t stride,
              int64_t batch_stride) {
  const auto fn = tensor_map_encoder();
  if (!fn) return false;
  const cuuint64_t gdim[3] = {(cuuint64_t)D, (cuuint64_t)q.T, (cuuint64_t)q.B};
  const cuuint64_t gstride[2] = {(cuuint64_t)stride * elt,
                                 (cuuint64_t)(q.B > 1 ? batch_stride : stride) * elt};
  const cuuint32_t box[3] = {CR_BOX, CR_STAGE, 1}, step[3] = {1, 1, 1};
  return fn(m, elt == 2 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_FLOAT32, 3,
            const_cast<void *>(base), gdim, gstride, box, step, CU_TENSOR_MAP_INTERLEAVE_NONE,
            CU_TENSOR_MAP_SWIZZLE_NONE, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
            CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// Runs of the ring: as long as let the whole call be on the GPU at once, whole
// stages.  Whether the ring serves a call: rows that TMA addresses, and enough of
// them that a block's start does not count (one prompt, 6144 channels, ring /
// simple kernel, us: forward the same up to 1024 tokens, two of 4096 41 / 55;
// gradient 512 tokens 10.4 / 12.9, 1024 14.8 / 19.1, 4096 37.5 / 110).
struct RingShape {
  bool use;
  int run, runs;
};
RingShape ring_shape(int32_t dtype, int B, int T, int D, bool bwd,
                     std::initializer_list<const void *> in, const void *out,
                     std::initializer_list<int64_t> in_strides,
                     std::initializer_list<int64_t> out_strides) {
  RingShape s{};
  const int elt = (int)dtype_bytes(dtype);
  const int channels =
      elt == 2 ? ConvRing<__nv_bfloat16, true>::CHANNELS : ConvRing<float, true>::CHANNELS;
  const int held = bwd ? ConvRing<float, true>::BLOCKS : ConvRing<float, false>::BLOCKS;
  const int64_t blocks = (D + channels - 1) / channels;
  const int64_t lanes = std::max<int64_t>(1, sm_count() * held / blocks / B);
  const int64_t run = ((T + lanes - 1) / lanes + CR_STAGE - 1) / CR_STAGE * CR_STAGE;
  s.use = whole_pieces(D, 4, dtype, {out}, out_strides) &&
          whole_pieces(16, 16 / elt, dtype, in, in_strides) && run >= CR_LEAST;
  s.run = (int)run;
  s.runs = s.use ? (int)((T + run - 1) / run) : 0;
  return s;
}

template <typename T, int W, bool BWD>
cudaError_t launch_ring(const void *grad, int64_t gs, int64_t gb, const ConvRingParams &p,
                        int64_t extra, cudaStream_t stream) {
  using R = ConvRing<T, BWD>;
  CUtensorMap x, g;
  if (!conv_map(&x, p.x, sizeof(T), p.q, p.D, p.xs, p.xb)) return cudaErrorInvalidValue;
  g = x;
  if (BWD && !conv_map(&g, grad, sizeof(T), p.q, p.D, gs, gb))
    return cudaErrorInvalidValue;
  constexpr int smem = R::STAGES * R::STAGE;
  const cudaError_t e = cudaFuncSetAttribute(
      conv_ring_kernel<T, W, BWD>, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
  if (e != cudaSuccess) return e;
  const dim3 grid((unsigned)((int64_t)p.q.B * p.runs + extra), (unsigned)((p.D + R::CHANNELS - 1) / R::CHANNELS));
  conv_ring_kernel<T, W, BWD><<<grid, R::THREADS + 32, smem, stream>>>(x, g, p);
  return cudaGetLastError();
}

gdn_status_t check_conv(int32_t dtype, int32_t w_dtype, int B, int T, int D, int W, int N,
                        int silu, const void *cu) {
  CHECK_DTYPE(dtype, "dtype");
  CHECK_DTYPE(w_dtype, "weight_dtype");
  CHECK_THAT(w_dtype == GDN_F32 || w_dtype == dtype, GDN_ERR_INVALID_ARG,
             "weight_dtype must be GDN_F32 or dtype");
  CHECK_THAT(B >= 1 && T >= 0 && D >= 1 && N >= 1, GDN_ERR_INVALID_ARG,
             "sizes must be positive (B=%d T=%d D=%d N=%d)", B, T, D, N);
  CHECK_THAT(W >= 2 && W <= 4, GDN_ERR_UNSUPPORTED, "W must be 2..4 (got %d)", W);
  CHECK_THAT(T <= MAX_TOKENS, GDN_ERR_UNSUPPORTED, "T (%d) must be at most %d", T, MAX_TOKENS);
  CHECK_FLAG(silu, "silu");
  if (cu == nullptr) {
    CHECK_THAT(N == B, GDN_ERR_INVALID_ARG, "without cu_seqlens N (%d) must equal B (%d)", N, B);
  } else {
    CHECK_THAT(B == 1, GDN_ERR_INVALID_ARG, "with cu_seqlens B must be 1 (got %d)", B);
    CHECK_OPT_PTR(cu, "cu_seqlens");
  }
  // one launch index counts the runs of all batch rows and the sequences
  CHECK_THAT((int64_t)B * (T / 4 + 1) + N <= 0x7fffffff, GDN_ERR_UNSUPPORTED,
             "B * T (%lld) is too long for one call", (long long)B * T);
  CHECK_THAT(D <= 32 * 65535, GDN_ERR_UNSUPPORTED, "D (%d) must be at most %d", D, 32 * 65535);
  return GDN_OK;
}

#define CHECK_STRIDE(s, name) \
  CHECK_THAT((s) >= a->D, GDN_ERR_INVALID_ARG, "%s (%lld) is less than D (%d)", name, (long long)(s), a->D)

// Shape of the gradient's launch: elements of a piece, tokens of a run and
// blocks along time.
struct BwdShape {
  bool ring = false;
  int vec, run, tiles;
  int64_t blocks;
};
BwdShape bwd_shape(const short_conv_bwd_args &a) {
  BwdShape s;
  const bool many = a.B > 1;
  const RingShape r =
      ring_shape(a.dtype, a.B, a.T, a.D, true, {a.dy, a.x}, a.dx,
                 {a.dy_stride, a.x_stride, many ? a.dy_batch_stride : 0,
                  many ? a.x_batch_stride : 0},
                 {a.dx_stride, many ? a.dx_batch_stride : 0});
  s.ring = r.use;
  if (r.use) {
    s.run = r.run;
    s.tiles = r.runs;
    s.blocks = (int64_t)a.B * r.runs;
    return s;
  }
  const int wide = CB_PIECE / 2;
  const bool whole = whole_pieces(a.D, wide, a.dtype, {a.dy, a.x, a.dx},
                                  {a.dy_stride, a.x_stride, a.dx_stride,
                                   many ? a.dy_batch_stride : 0, many ? a.x_batch_stride : 0,
                                   many ? a.dx_batch_stride : 0});
  s.vec = whole ? wide : 1;
  s.run = run_tokens((int64_t)a.B * a.T, (a.D + s.vec - 1) / s.vec, 32 * CB_RUNS * CB_BLOCKS);
  if (s.run < 8) s.run = 8;
  const int64_t span = (int64_t)s.run * CB_RUNS;
  s.tiles = (int)((a.T + span - 1) / span);
  s.blocks = (int64_t)a.B * s.tiles;
  return s;
}

}  // namespace
}  // namespace gdn

using namespace gdn;

extern "C" {

gdn_status_t short_conv_fwd(const short_conv_args *a, gdn_stream_t stream) {
  (void)set_host_error(GDN_OK, "");
  CHECK_THAT(a != nullptr, GDN_ERR_INVALID_ARG, "args is NULL");
  gdn_status_t st = check_conv(a->dtype, a->weight_dtype, a->B, a->T, a->D, a->W, a->N, a->silu,
                               a->cu_seqlens);
  if (st != GDN_OK) return st;
  if (a->T > 0) {
    CHECK_TOKENS(a->x, "x", a->dtype);
    CHECK_TOKENS(a->y, "y", a->dtype);
    CHECK_STRIDE(a->x_stride, "x_stride");
    CHECK_STRIDE(a->y_stride, "y_stride");
  }
  CHECK_PTR(a->weight, "weight");
  CHECK_OPT_PTR(a->bias, "bias");
  CHECK_OPT_PTR(a->h0, "h0");
  CHECK_OPT_PTR(a->ht, "ht");
  ConvParams p{};
  p.x = a->x; p.weight = a->weight; p.bias = a->bias; p.h0 = a->h0; p.ht = a->ht; p.y = a->y;
  p.q = {a->cu_seqlens, a->B, a->T, a->N};
  p.xs = a->x_stride; p.xb = a->B > 1 ? a->x_batch_stride : 0;
  p.ys = a->y_stride; p.yb = a->B > 1 ? a->y_batch_stride : 0;
  p.D = a->D; p.silu = a->silu; p.w_f32 = a->weight_dtype == GDN_F32;
  const RingShape r = ring_shape(a->dtype, a->B, a->T, a->D, false, {a->x}, a->y, {p.xs, p.xb},
                                 {p.ys, p.yb});
  const int wide = CV_PIECE / 2;
  const bool whole = whole_pieces(a->D, wide, a->dtype, {a->x, a->y}, {p.xs, p.xb, p.ys, p.yb});
  const int64_t pieces = a->D / (whole ? wide : 1);
  p.run = run_tokens((int64_t)a->B * a->T, pieces, CV_MAX_THREADS * CV_BLOCKS);
  p.tiles = (int)(((int64_t)a->T + p.run - 1) / p.run);
  const int block = even_block(pieces);
  const int64_t gx = (int64_t)a->B * p.tiles + (a->ht ? a->N : 0);
  if (gx == 0) return GDN_OK;
  p.err = device_error_word();
  if (p.err == nullptr) return launch_status(cudaGetLastError(), "device error word");
  if (r.use) {
    ConvRingParams rp{};
    rp.weight = a->weight; rp.bias = a->bias; rp.h0 = a->h0; rp.out = a->y; rp.ht = a->ht;
    rp.err = p.err; rp.q = p.q; rp.xs = p.xs; rp.xb = p.xb; rp.os = p.ys; rp.ob = p.yb;
    rp.x = a->x; rp.D = p.D; rp.silu = p.silu; rp.w_f32 = p.w_f32;
    rp.run = r.run; rp.runs = r.runs;
    return launch_status(with_types(a->dtype, a->W,
                                    [&](auto t, auto w) {
                                      return launch_ring<decltype(t), decltype(w)::value, false>(
                                          nullptr, 0, 0, rp, a->ht ? a->N : 0,
                                          reinterpret_cast<cudaStream_t>(stream));
                                    }),
                         "short convolution launch");
  }
  const dim3 grid((unsigned)gx, (unsigned)((pieces + block - 1) / block));
  return launch_status(
      with_types(a->dtype, a->W,
                 [&](auto t, auto w) {
                   using T = decltype(t);
                   constexpr int W = decltype(w)::value;
                   cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
                   if (whole)
                     conv_fwd_kernel<T, CV_PIECE / 2, W><<<grid, block, 0, s>>>(p);
                   else
                     conv_fwd_kernel<T, 1, W><<<grid, block, 0, s>>>(p);
                   return cudaGetLastError();
                 }),
      "short convolution launch");
}

gdn_status_t short_conv_bwd_workspace_size(const short_conv_bwd_args *a, size_t *bytes) {
  CHECK_THAT(a != nullptr && bytes != nullptr, GDN_ERR_INVALID_ARG, "NULL argument");
  *bytes = 0;
  gdn_status_t st = check_conv(a->dtype, a->weight_dtype, a->B, a->T, a->D, a->W, a->N, a->silu,
                               a->cu_seqlens);
  if (st != GDN_OK) return st;
  if (a->dweight || a->dbias)
    *bytes = (size_t)bwd_shape(*a).blocks * (a->W + 1) * a->D * sizeof(float);
  return GDN_OK;
}

gdn_status_t short_conv_bwd(const short_conv_bwd_args *a, gdn_stream_t stream) {
  (void)set_host_error(GDN_OK, "");
  CHECK_THAT(a != nullptr, GDN_ERR_INVALID_ARG, "args is NULL");
  gdn_status_t st = check_conv(a->dtype, a->weight_dtype, a->B, a->T, a->D, a->W, a->N, a->silu,
                               a->cu_seqlens);
  if (st != GDN_OK) return st;
  if (a->T > 0) {
    CHECK_TOKENS(a->dy, "dy", a->dtype);
    CHECK_TOKENS(a->x, "x", a->dtype);
    CHECK_TOKENS(a->dx, "dx", a->dtype);
    CHECK_STRIDE(a->dy_stride, "dy_stride");
    CHECK_STRIDE(a->x_stride, "x_stride");
    CHECK_STRIDE(a->dx_stride, "dx_stride");
  }
  CHECK_PTR(a->weight, "weight");
  CHECK_OPT_PTR(a->bias, "bias");
  CHECK_OPT_PTR(a->h0, "h0");
  CHECK_OPT_PTR(a->dht, "dht");
  CHECK_OPT_PTR(a->dh0, "dh0");
  CHECK_OPT_PTR(a->dweight, "dweight");
  CHECK_OPT_PTR(a->dbias, "dbias");
  const BwdShape shape = bwd_shape(*a);
  const bool sums = a->dweight || a->dbias;
  if (sums && shape.blocks > 0) {
    const size_t need = (size_t)shape.blocks * (a->W + 1) * a->D * sizeof(float);
    CHECK_THAT(a->workspace != nullptr && a->workspace_bytes >= need, GDN_ERR_WORKSPACE,
               "workspace of %zu bytes needed (got %zu)", need, a->workspace_bytes);
    CHECK_OPT_PTR(a->workspace, "workspace");
  }
  ConvBwdParams p{};
  p.dy = a->dy; p.x = a->x; p.weight = a->weight; p.bias = a->bias; p.h0 = a->h0; p.dht = a->dht;
  p.dx = a->dx; p.dh0 = a->dh0;
  p.part = sums ? static_cast<float *>(a->workspace) : nullptr;
  p.q = {a->cu_seqlens, a->B, a->T, a->N};
  p.gs = a->dy_stride; p.gb = a->B > 1 ? a->dy_batch_stride : 0;
  p.xs = a->x_stride; p.xb = a->B > 1 ? a->x_batch_stride : 0;
  p.ds = a->dx_stride; p.db = a->B > 1 ? a->dx_batch_stride : 0;
  p.D = a->D; p.silu = a->silu; p.w_f32 = a->weight_dtype == GDN_F32;
  p.run = shape.run; p.tiles = shape.tiles;
  p.err = device_error_word();
  if (p.err == nullptr) return launch_status(cudaGetLastError(), "device error word");
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  auto sum_parts = [&](auto w) {
    constexpr int W = decltype(w)::value;
    if (sums)
      conv_bwd_sum_kernel<W><<<dim3((a->D + 31) / 32, W + 1), dim3(32, 8), 0, s>>>(
          p.part, (int)shape.blocks, a->D, a->dweight, a->dbias, p.q, p.err);
    return cudaGetLastError();
  };
  if (shape.ring) {
    ConvRingParams r{};
    r.weight = a->weight; r.bias = a->bias; r.h0 = a->h0; r.dht = a->dht;
    r.out = a->dx; r.ht = a->dh0; r.part = p.part; r.err = p.err; r.q = p.q;
    r.xs = p.xs; r.xb = p.xb; r.os = p.ds; r.ob = p.db; r.x = a->x;
    r.D = p.D; r.silu = p.silu; r.w_f32 = p.w_f32; r.run = shape.run; r.runs = shape.tiles;
    return launch_status(
        with_types(a->dtype, a->W,
                   [&](auto t, auto w) {
                     const cudaError_t e = launch_ring<decltype(t), decltype(w)::value, true>(
                         a->dy, p.gs, p.gb, r, a->dh0 ? a->N : 0, s);
                     return e != cudaSuccess ? e : sum_parts(w);
                   }),
        "short convolution gradient launch");
  }
  const int64_t gx = shape.blocks + (a->dh0 ? a->N : 0);
  const dim3 grid((unsigned)gx, (unsigned)((a->D + 32 * shape.vec - 1) / (32 * shape.vec)));
  return launch_status(
      with_types(a->dtype, a->W,
                 [&](auto t, auto w) {
                   using T = decltype(t);
                   constexpr int W = decltype(w)::value;
                   const dim3 block(32, CB_RUNS);
                   if (gx > 0) {
                     if (shape.vec > 1)
                       conv_bwd_kernel<T, CB_PIECE / 2, W><<<grid, block, 0, s>>>(p);
                     else
                       conv_bwd_kernel<T, 1, W><<<grid, block, 0, s>>>(p);
                     const cudaError_t e = cudaGetLastError();
                     if (e != cudaSuccess) return e;
                   }
                   return sum_parts(w);
                 }),
      "short convolution gradient launch");
}

gdn_status_t short_conv_decode(const short_conv_decode_args *a, gdn_stream_t stream) {
  (void)set_host_error(GDN_OK, "");
  CHECK_THAT(a != nullptr, GDN_ERR_INVALID_ARG, "args is NULL");
  CHECK_THAT(a->T >= 1 && a->T <= 4, GDN_ERR_UNSUPPORTED, "T must be 1..4 (got %d)", a->T);
  gdn_status_t st = check_conv(a->dtype, a->weight_dtype, a->B, a->T, a->D, a->W, a->B, a->silu,
                               nullptr);
  if (st != GDN_OK) return st;
  CHECK_THAT(a->pool >= 1, GDN_ERR_INVALID_ARG, "pool must be positive (got %d)", a->pool);
  CHECK_THAT(a->slot_indices != nullptr || a->pool >= a->B, GDN_ERR_INVALID_ARG,
             "identity slots need pool (%d) >= B (%d)", a->pool, a->B);
  CHECK_TOKENS(a->x, "x", a->dtype);
  CHECK_TOKENS(a->y, "y", a->dtype);
  CHECK_STRIDE(a->x_stride, "x_stride");
  CHECK_STRIDE(a->y_stride, "y_stride");
  CHECK_PTR(a->weight, "weight");
  CHECK_OPT_PTR(a->bias, "bias");
  CHECK_PTR(a->state, "state");
  CHECK_OPT_PTR(a->slot_indices, "slot_indices");
  ConvDecodeParams p{};
  p.x = a->x; p.weight = a->weight; p.bias = a->bias; p.state = a->state; p.y = a->y;
  p.slots = a->slot_indices;
  p.xs = a->x_stride; p.xb = a->B > 1 ? a->x_batch_stride : 0;
  p.ys = a->y_stride; p.yb = a->B > 1 ? a->y_batch_stride : 0;
  p.B = a->B; p.T = a->T; p.D = a->D; p.pool = a->pool; p.silu = a->silu;
  p.w_f32 = a->weight_dtype == GDN_F32;
  p.err = device_error_word();
  if (p.err == nullptr) return launch_status(cudaGetLastError(), "device error word");
  const int wide = 16 / (int)dtype_bytes(a->dtype);
  const bool whole = whole_pieces(a->D, wide, a->dtype, {a->x, a->y}, {p.xs, p.xb, p.ys, p.yb});
  const int64_t pieces = a->D / (whole ? wide : 1);
  const int block = even_block(pieces);
  const dim3 grid((unsigned)a->B, (unsigned)((pieces + block - 1) / block));
  return launch_status(
      with_types(a->dtype, a->W,
                 [&](auto t, auto w) {
                   using T = decltype(t);
                   constexpr int W = decltype(w)::value;
                   cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
                   if (whole)
                     conv_decode_kernel<T, 16 / sizeof(T), W><<<grid, block, 0, s>>>(p);
                   else
                     conv_decode_kernel<T, 1, W><<<grid, block, 0, s>>>(p);
                   return cudaGetLastError();
                 }),
      "short convolution token launch");
}

}  // extern "C"
