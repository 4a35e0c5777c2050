// The gated delta rule's gradient over chunks on CUDA cores, in float32 throughout: every
// call that the tensor cores do not take (float32, odd head sizes, V > 128).  delta_bwd.h has
// the formulas.
//
// All products go through one tiled product of a block: 64 x 64 outputs, 16 of them a thread,
// of which half of the threads sum every other 16 steps; operands are read through functions,
// so that gates, masks and transposes need no copies.  What bounds a call of few heads is the
// latency of the products that wait for one another along a walk, half of it instructions: the
// next 32 steps' operands are on their way in registers while 32 are multiplied, and every
// load is of a place that exists, with the value chosen behind it, so that no load waits for
// another.  (Three sequences of 261 to 376 tokens, 12 heads of 48 x 40, float32: 323 us; a
// thread summing all steps, 256 of them, 353 (then 320); with 16 steps a tile, two barriers each, and loads
// inside branches 502.  A walk's rows and state kept in shared memory instead of the workspace
// changed nothing.)
#include "delta_bwd.h"
#include "gdn_common.cuh"
#include "ptx.cuh"
#include "rows.cuh"

namespace gdn {
namespace {

constexpr int Q = 64, THREADS = 512, COLS = 64;
constexpr int DEPTH = 32, TILE = DEPTH * (Q + 4);  // steps and floats of one operand's tile
constexpr int TILES = 4 * TILE;      // two operands, two buffers
constexpr int SIDE = Q + 1;          // pitch of square matrices in shared memory

// A chunk and head's floats: running log-gates and beta, T, P, n and dr [64][V], the state
// and its gradient [K][V].  T is read as a lower triangle; above it, in the last columns of its
// first two rows, lies what the gates' rounding left.
struct Block {
  float *G, *beta, *T, *P, *n, *dr, *h, *D;
  __device__ Block(const DeltaBwdParams &p, int64_t chunk, int head) {
    float *f = reinterpret_cast<float *>(p.blocks + (chunk * p.H + head) * p.block);
    G = f;
    beta = G + Q;
    T = beta + Q;
    P = T + Q * Q;
    n = P + Q * Q;
    dr = n + (int64_t)Q * p.V;
    h = dr + (int64_t)Q * p.V;
    D = h + (int64_t)p.K * p.V;
  }
  __device__ __forceinline__ float &rest(int i) const { return T[i / 32 * Q + 32 + i % 32]; }
  __device__ __forceinline__ float lower(int i, int j) const {
    const float x = T[i * Q + j];
    return i >= j ? x : 0.f;
  }
};

int64_t block_floats(const DeltaBwdParams &p) {
  return 2 * Q + 2 * Q * Q + 2 * (int64_t)(Q + p.K) * p.V;
}

// Which of an operand's indexes neighbouring threads take: the one along which it is stored.
enum Along { ROWS, STEPS };  // (a's rows and b's columns; or the steps of the sum)

template <Along ALONG>
__device__ __forceinline__ void tile_place(int e, int &row, int &step) {
  const int tid = threadIdx.x;
  if (ALONG == STEPS) {  // eight steps of four rows a warp: whole sectors, no bank twice
    step = tid % 8 + 8 * e;
    row = tid / 8;
  } else {
    row = tid % 64;
    step = tid / 64 + 8 * e;
  }
}

// out(i, j, sum_k a(i, k) b(k, j)) for i < M, j < N; a and b are only asked for what is inside.
// `tiles` is shared memory of TILES floats.  Every operand is read before the first output of
// its 64 x 64 tile is written.
template <Along A_ALONG, Along B_ALONG, typename A, typename B, typename Out>
__device__ __forceinline__ void product(int M, int N, int K, float *tiles, A a, B b, Out out) {
  constexpr int EACH = DEPTH * Q / THREADS, PITCH = Q + 4;
  const int half = threadIdx.x / 256, ti = threadIdx.x % 256 / 16 * 4, tj = threadIdx.x % 16 * 4;
  for (int i0 = 0; i0 < M; i0 += 64)
    for (int j0 = 0; j0 < N; j0 += 64) {
      float acc[4][4] = {}, x[EACH], y[EACH];
      auto fetch = [&](int k0) {
#pragma unroll
        for (int e = 0; e < EACH; ++e) {
          int r, k;
          tile_place<A_ALONG>(e, r, k);
          const float u = a(min(i0 + r, M - 1), min(k0 + k, K - 1));
          x[e] = i0 + r < M && k0 + k < K ? u : 0.f;
          tile_place<B_ALONG>(e, r, k);
          const float v = b(min(k0 + k, K - 1), min(j0 + r, N - 1));
          y[e] = j0 + r < N && k0 + k < K ? v : 0.f;
        }
      };
      fetch(0);
      for (int k0 = 0, turn = 0; k0 < K; k0 += DEPTH, turn ^= 1) {
        float *as = tiles + turn * 2 * TILE, *bs = as + TILE;
#pragma unroll
        for (int e = 0; e < EACH; ++e) {
          int r, k;
          tile_place<A_ALONG>(e, r, k);
          as[k * PITCH + r] = x[e];
          tile_place<B_ALONG>(e, r, k);
          bs[k * PITCH + r] = y[e];
        }
        __syncthreads();
        if (k0 + DEPTH < K) fetch(k0 + DEPTH);
        const int steps = min((half + 1) * DEPTH / 2, K - k0);
#pragma unroll 8
        for (int k = half * DEPTH / 2; k < steps; ++k) {
          const float4 u = *reinterpret_cast<const float4 *>(as + k * PITCH + ti);
          const float4 v = *reinterpret_cast<const float4 *>(bs + k * PITCH + tj);
          const float f[4] = {u.x, u.y, u.z, u.w}, g[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const float both[4] = {f[i], f[i], f[i], f[i]};
            fma_row<4>(acc[i], both, g);
          }
        }
      }
      __syncthreads();  // the tiles have been read
      // each half is left with two of a thread's rows
      float *other = tiles + (threadIdx.x ^ 256);
#pragma unroll
      for (int i = 0; i < 2; ++i)
#pragma unroll
        for (int j = 0; j < 4; ++j) tiles[(4 * i + j) * THREADS + threadIdx.x] = half ? acc[i][j] : acc[i + 2][j];
      __syncthreads();
#pragma unroll
      for (int i = 0; i < 2; ++i)
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const int row = i0 + ti + i + 2 * half, col = j0 + tj + j;
          const float sum = (half ? acc[i + 2][j] : acc[i][j]) + other[(4 * i + j) * THREADS];
          if (row < M && col < N) out(row, col, sum);
        }
      __syncthreads();
    }
}

// Rows of a token tensor [.., heads, D] of one chunk and head; zero past its end.
template <typename E>
struct Rows {
  const E *at;
  int64_t stride;
  int len;
  __device__ Rows(const void *base, int64_t token, int heads, int head, int D, int len_)
      : at(static_cast<const E *>(base) + (token * heads + head) * D), stride((int64_t)heads * D),
        len(len_) {}
  __device__ float operator()(int i, int c) const {
    const float x = to_f32(at[min(i, len - 1) * stride + c]);
    return i < len ? x : 0.f;
  }
};

// grid: chunks, heads.  G, beta, P, A and T = (I + A)^-1: its 16 x 16 blocks on the diagonal by
// forward substitution, a column a thread, then the blocks below, a diagonal at a time,
// T_(b+d, b) = -T_(b+d, b+d) sum_m A_(b+d, m) T_(m, b).  (All 64 rows by substitution, unrolled,
// are 40 KB of instructions that wait to be fetched.)
template <typename E>
__global__ void __launch_bounds__(THREADS) simt_prepare_kernel(DeltaBwdParams p) {
  extern __shared__ __align__(16) float shared[];
  __shared__ float G[Q], beta[Q], rest[Q];
  float *tiles = shared, *A = shared + TILES;  // [Q][SIDE]
  ptx::griddep_wait();
  const DeltaChunk ch = delta_chunk(p, blockIdx.x);
  const int head = blockIdx.y, hk = head / (p.H / p.Hg), tid = threadIdx.x;
  if (ch.len <= 0) return;
  if (!bounds_ok(ch.n < p.N && ch.token + ch.len <= (int64_t)p.B * p.T, p.err)) return;
  const Block w(p, blockIdx.x, head);
  if (tid < Q) {
    const int64_t at = (ch.token + min(tid, ch.len - 1)) * p.H + head;
    G[tid] = tid < ch.len || p.g_is_cumsum ? p.g[at] : 0.f;
    if (!p.g_is_cumsum) G[tid] = delta_gate(G[tid]);
    beta[tid] = tid < ch.len ? p.beta[at] : 0.f;
    rest[tid] = 0.f;
  }
  __syncthreads();
  if (tid < 32 && !p.g_is_cumsum) {  // (one thread after another, in 64 bits: 30 us more)
    double sum[2] = {G[tid], G[tid + 32]};
#pragma unroll
    for (int e = 0; e < 2; ++e)
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const double x = __shfl_up_sync(~0u, sum[e], o);
        if (tid >= o) sum[e] += x;
      }
    sum[1] += __shfl_sync(~0u, sum[0], 31);
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      const float f = (float)sum[e];
      G[tid + 32 * e] = f;
      rest[tid + 32 * e] = (float)(sum[e] - f);
    }
  }
  __syncthreads();
  if (tid < Q) {
    w.G[tid] = G[tid];
    w.beta[tid] = beta[tid];
  }
  const Rows<E> q(p.q, ch.token, p.Hg, hk, p.K, ch.len), k(p.k, ch.token, p.Hg, hk, p.K, ch.len);
  auto kt = [&](int c, int j) { return k(j, c); };
  product<STEPS, STEPS>(Q, Q, p.K, tiles, q, kt, [&](int i, int j, float s) {
    w.P[i * Q + j] = i >= j ? p.scale * s * expf(delta_gap(G[i], rest[i], G[j], rest[j])) : 0.f;
  });
  product<STEPS, STEPS>(Q, Q, p.K, tiles, k, kt, [&](int i, int j, float s) {
    A[i * SIDE + j] = i > j ? beta[i] * s * expf(delta_gap(G[i], rest[i], G[j], rest[j])) : 0.f;
  });
  float *T = tiles, *Y = tiles + Q * SIDE;  // (A's products are through)
  for (int x = tid; x < Q * Q; x += THREADS) T[x / Q * SIDE + x % Q] = 0.f;
  __syncthreads();
  if (tid < Q) {
    const int b = tid / 16 * 16, j = tid % 16;
    float x[16];
#pragma unroll
    for (int i = 0; i < 16; ++i) {
      x[i] = i == j ? 1.f : 0.f;
#pragma unroll
      for (int m = 0; m < i; ++m) x[i] = fmaf(-A[(b + i) * SIDE + b + m], x[m], x[i]);
      T[(b + i) * SIDE + tid] = x[i];
    }
  }
  __syncthreads();
  for (int d = 16; d < Q; d += 16) {
    for (int x = tid; x < (Q - d) * 16; x += THREADS) {
      const int col = x % (Q - d), b = col / 16 * 16, row = b + d + x / (Q - d);
      float v = 0.f;
      for (int m = b; m < b + d; ++m) v = fmaf(A[row * SIDE + m], T[m * SIDE + col], v);
      Y[row * SIDE + col] = v;
    }
    __syncthreads();
    for (int x = tid; x < (Q - d) * 16; x += THREADS) {
      const int col = x % (Q - d), b = col / 16 * 16 + d, row = b + x / (Q - d);
      float v = 0.f;
      for (int m = b; m < b + 16; ++m) v = fmaf(-T[row * SIDE + m], Y[m * SIDE + col], v);
      T[row * SIDE + col] = v;
    }
    __syncthreads();
  }
  for (int x = tid; x < Q * Q; x += THREADS) {
    const int i = x / Q, j = x % Q;
    w.T[x] = i < 2 && j >= 32 ? rest[i * 32 + j - 32] : T[i * SIDE + j];
  }
}

// The factors of a chunk's rows in a walk: beta, e^G and e^(G_L - G), which is zero past the
// chunk's end (there the gate may not be a sum).
struct Factors {
  float beta[Q], eG[Q], eR[Q];
  __device__ __forceinline__ void load(const Block &w, int len) {
    __syncthreads();  // the ones before have been read
    if (threadIdx.x < Q) {
      const int i = threadIdx.x;
      const float G = w.G[i], R = delta_gap(w.G[len - 1], w.rest(len - 1), G, w.rest(i));
      beta[i] = w.beta[i];
      eG[i] = expf(G);
      eR[i] = i < len ? expf(R) : 0.f;
    }
    __syncthreads();
  }
};

// grid: 64 value columns, heads, sequences.  The states, forward.
template <typename E>
__global__ void __launch_bounds__(THREADS) simt_states_kernel(DeltaBwdParams p) {
  __shared__ __align__(16) float tiles[TILES];
  __shared__ Factors f;
  const int v0 = blockIdx.x * COLS, nv = min(COLS, p.V - v0), head = blockIdx.y;
  const int hk = head / (p.H / p.Hg), K = p.K, V = p.V;
  int64_t first;
  ptx::griddep_wait();
  if (!delta_good(p)) return;
  const int n = delta_turn(p, blockIdx.z), count = delta_chunks(p, n, &first);
  if (count == 0) return;
  {
    const Block w(p, first, head);
    const int64_t state = ((int64_t)n * p.H + head) * K * V;
    for (int x = threadIdx.x; x < K * nv; x += THREADS) {
      const int c = x / nv, j = v0 + x % nv;
      const int64_t at = state + (p.v_first ? (int64_t)j * K + c : (int64_t)c * V + j);
      w.h[(int64_t)c * V + j] = p.h0 ? p.h0[at] : 0.f;
    }
    __syncthreads();
  }
  for (int c = 0; c < count; ++c) {
    const DeltaChunk ch = delta_chunk(p, first + c);
    const Block w(p, first + c, head);
    const Rows<E> k(p.k, ch.token, p.Hg, hk, K, ch.len), v(p.v, ch.token, p.H, head, V, ch.len);
    f.load(w, ch.len);
    product<STEPS, ROWS>(Q, nv, K, tiles, k, [&](int i, int j) { return w.h[(int64_t)i * V + v0 + j]; },
                         [&](int i, int j, float s) {
                           w.n[(int64_t)i * V + v0 + j] = f.beta[i] * (v(i, v0 + j) - f.eG[i] * s);
                         });
    auto rows = [&](int i, int j) { return w.n[(int64_t)i * V + v0 + j]; };
    product<STEPS, ROWS>(Q, nv, Q, tiles, [&](int i, int m) { return w.lower(i, m); }, rows,
                         [&](int i, int j, float s) { w.n[(int64_t)i * V + v0 + j] = s; });
    if (c + 1 == count) break;
    const Block next(p, first + c + 1, head);
    const float keep = f.eG[ch.len - 1];
    product<ROWS, ROWS>(K, nv, ch.len, tiles, [&](int kc, int i) { return k(i, kc) * f.eR[i]; }, rows,
                        [&](int kc, int j, float s) {
                          const int64_t at = (int64_t)kc * V + v0 + j;
                          next.h[at] = fmaf(keep, w.h[at], s);
                        });
  }
}

// grid: as simt_states_kernel.  The states' gradients, backward.
template <typename E>
__global__ void __launch_bounds__(THREADS) simt_grads_kernel(DeltaBwdParams p) {
  __shared__ __align__(16) float tiles[TILES];
  __shared__ Factors f;
  const int v0 = blockIdx.x * COLS, nv = min(COLS, p.V - v0), head = blockIdx.y;
  const int hk = head / (p.H / p.Hg), K = p.K, V = p.V;
  int64_t first;
  ptx::griddep_wait();
  if (!delta_good(p)) return;
  const int n = delta_turn(p, blockIdx.z), count = delta_chunks(p, n, &first);
  const int64_t state = ((int64_t)n * p.H + head) * K * V;
  auto outer = [&](int c, int j) {  // of h0, dht and dh0
    return state + (p.v_first ? (int64_t)j * K + c : (int64_t)c * V + j);
  };
  for (int x = threadIdx.x; x < K * nv; x += THREADS) {
    const int c = x / nv, j = v0 + x % nv;
    const float d = p.dht ? p.dht[outer(c, j)] : 0.f;
    if (count > 0)
      Block(p, first + count - 1, head).D[(int64_t)c * V + j] = d;
    else if (p.dh0)
      p.dh0[outer(c, j)] = d;
  }
  __syncthreads();
  for (int c = count - 1; c >= 0; --c) {
    const DeltaChunk ch = delta_chunk(p, first + c);
    const Block w(p, first + c, head);
    const Rows<E> q(p.q, ch.token, p.Hg, hk, K, ch.len), k(p.k, ch.token, p.Hg, hk, K, ch.len);
    const Rows<E> go(p.dout, ch.token, p.H, head, V, ch.len);
    f.load(w, ch.len);
    const float keep = f.eG[ch.len - 1];
    product<ROWS, ROWS>(Q, nv, Q, tiles, [&](int j, int i) { return w.P[i * Q + j]; },
                        [&](int i, int j) { return go(i, v0 + j); },
                        [&](int i, int j, float s) { w.dr[(int64_t)i * V + v0 + j] = s; });
    product<STEPS, ROWS>(Q, nv, K, tiles, k, [&](int i, int j) { return w.D[(int64_t)i * V + v0 + j]; },
                         [&](int i, int j, float s) { w.dr[(int64_t)i * V + v0 + j] += f.eR[i] * s; });
    auto rows = [&](int i, int j) { return w.dr[(int64_t)i * V + v0 + j]; };
    product<ROWS, ROWS>(Q, nv, Q, tiles, [&](int i, int m) { return w.lower(m, i); }, rows,
                        [&](int i, int j, float s) { w.dr[(int64_t)i * V + v0 + j] = s; });
    if (c == 0 && p.dh0 == nullptr) break;
    float *prev = c > 0 ? Block(p, first + c - 1, head).D : nullptr;
    // steps 0 .. 63: q and do, behind them k and dr
    product<ROWS, ROWS>(K, nv, 2 * Q, tiles,
                        [&](int kc, int i) {
                          const Rows<E> &from = i < Q ? q : k;
                          const float x = from(i % Q, kc) * f.eG[i % Q];
                          return i < Q ? p.scale * x : -f.beta[i % Q] * x;
                        },
                        [&](int i, int j) {
                          const float x = go(i % Q, v0 + j), y = rows(i % Q, j);
                          return i < Q ? x : y;
                        },
                        [&](int kc, int j, float s) {
                          const float d = fmaf(keep, w.D[(int64_t)kc * V + v0 + j], s);
                          if (prev)
                            prev[(int64_t)kc * V + v0 + j] = d;
                          else
                            p.dh0[outer(kc, v0 + j)] = d;
                        });
  }
}

// Shared memory of simt_inputs_kernel, in floats.
struct Inputs {
  float *tiles, *dq, *dk, *x, *P, *A, *M, *B, *sums;
  __device__ explicit Inputs(float *f) {
    tiles = f;
    dq = tiles + TILES;
    dk = dq + Q * KMAX;
    x = dk + Q * KMAX;
    P = x + Q * KMAX;
    A = P + Q * SIDE;
    M = A + Q * SIDE;
    B = M + Q * SIDE;
    sums = B + Q * SIDE;   // 8 x 64
  }
  static constexpr int FLOATS = TILES + 3 * Q * KMAX + 4 * Q * SIDE + 8 * Q;
};

constexpr int EACH_ROW = THREADS / Q;  // threads of a row
// v over a row's threads.
__device__ __forceinline__ float row_sum(float v) {
#pragma unroll
  for (int o = 1; o < EACH_ROW; o <<= 1) v += __shfl_xor_sync(~0u, v, o);
  return v;
}

// sum_c x[i][c] y(i, c) of every row to out[i].
template <typename Y>
__device__ __forceinline__ void row_dots(const float *x, int K, Y y, float *out) {
  const int i = threadIdx.x / EACH_ROW;
  float s = 0.f;
  for (int c = threadIdx.x % EACH_ROW; c < K; c += EACH_ROW) s = fmaf(x[i * K + c], y(i, c), s);
  s = row_sum(s);
  if (threadIdx.x % EACH_ROW == 0) out[i] = s;
  __syncthreads();
}

// grid: chunks, key heads.  The gradients of a chunk's tokens; the value heads of a key head
// one after another, their dq and dk summed in shared memory.
template <typename E>
__global__ void __launch_bounds__(THREADS) simt_inputs_kernel(DeltaBwdParams p) {
  extern __shared__ __align__(16) float shared[];
  __shared__ Factors f;
  const Inputs s(shared);
  ptx::griddep_wait();
  const DeltaChunk ch = delta_chunk(p, blockIdx.x);
  const int hk = blockIdx.y, rep = p.H / p.Hg, tid = threadIdx.x, K = p.K, V = p.V;
  if (ch.len <= 0) return;
  if (!bounds_ok(ch.n < p.N && ch.token + ch.len <= (int64_t)p.B * p.T, p.err)) return;
  const Rows<E> q(p.q, ch.token, p.Hg, hk, K, ch.len), k(p.k, ch.token, p.Hg, hk, K, ch.len);
  float *qd = s.sums, *kh = qd + Q, *kD = kh + Q, *G = kD + Q, *dG = G + Q, *rest = dG + Q;
  float *part = rest + Q;
  for (int x = tid; x < Q * K; x += THREADS) s.dq[x] = s.dk[x] = 0.f;
  __syncthreads();
  for (int head = hk * rep; head < (hk + 1) * rep; ++head) {
    const Block w(p, blockIdx.x, head);
    const Rows<E> go(p.dout, ch.token, p.H, head, V, ch.len), v(p.v, ch.token, p.H, head, V, ch.len);
    f.load(w, ch.len);
    const float keep = f.eG[ch.len - 1];
    if (tid < Q) {
      G[tid] = w.G[tid];
      rest[tid] = w.rest(tid);
    }
    __syncthreads();
    auto kt = [&](int c, int j) { return k(j, c); };
    auto n = [&](int i, int c) { return w.n[(int64_t)i * V + c]; };
    auto nt = [&](int c, int j) { return n(j, c); };
    auto dr = [&](int i, int c) { return w.dr[(int64_t)i * V + c]; };
    auto ht = [&](int c, int kc) { return w.h[(int64_t)kc * V + c]; };
    auto Dt = [&](int c, int kc) { return w.D[(int64_t)kc * V + c]; };
    product<STEPS, STEPS>(Q, Q, K, s.tiles, q, kt, [&](int i, int j, float x) { s.P[i * SIDE + j] = x; });
    product<STEPS, STEPS>(Q, Q, V, s.tiles, go, nt, [&](int i, int j, float x) {
      const bool in = i >= j && i < ch.len;
      const float L = in ? p.scale * expf(delta_gap(G[i], rest[i], G[j], rest[j])) : 0.f;
      s.M[i * SIDE + j] = i > j ? L * x * s.P[i * SIDE + j] : 0.f;
      s.P[i * SIDE + j] = L * x;
    });
    product<STEPS, STEPS>(Q, Q, K, s.tiles, k, kt, [&](int i, int j, float x) { s.A[i * SIDE + j] = x; });
    product<STEPS, STEPS>(Q, Q, V, s.tiles, dr, nt, [&](int i, int j, float x) {
      const bool in = i > j && i < ch.len;
      const float L = in ? expf(delta_gap(G[i], rest[i], G[j], rest[j])) : 0.f;
      s.B[i * SIDE + j] = -L * x * s.A[i * SIDE + j];
      s.A[i * SIDE + j] = -L * x * f.beta[i];
    });
    product<STEPS, STEPS>(Q, K, V, s.tiles, go, ht, [&](int i, int c, float x) {
      x *= p.scale * f.eG[i];
      s.x[i * K + c] = x;
      s.dq[i * K + c] += x;
    });
    row_dots(s.x, K, q, qd);
    product<STEPS, STEPS>(Q, K, V, s.tiles, dr, ht, [&](int i, int c, float x) {
      x *= -f.eG[i];
      s.x[i * K + c] = x;
      s.dk[i * K + c] += f.beta[i] * x;
    });
    row_dots(s.x, K, k, kh);
    product<STEPS, STEPS>(Q, K, V, s.tiles, n, Dt, [&](int i, int c, float x) {
      x *= f.eR[i];
      s.x[i * K + c] = x;
      s.dk[i * K + c] += x;
    });
    row_dots(s.x, K, k, kD);
    product<STEPS, ROWS>(Q, K, Q, s.tiles, [&](int i, int j) { return s.P[i * SIDE + j]; }, k,
                         [&](int i, int c, float x) { s.dq[i * K + c] += x; });
    product<ROWS, ROWS>(Q, K, Q, s.tiles, [&](int j, int i) { return s.P[i * SIDE + j]; }, q,
                        [&](int i, int c, float x) { s.dk[i * K + c] += x; });
    product<STEPS, ROWS>(Q, K, Q, s.tiles,
                         [&](int i, int j) { return s.A[i * SIDE + j] + s.A[j * SIDE + i]; }, k,
                         [&](int i, int c, float x) { s.dk[i * K + c] += x; });
    // dr.v of every row, and dv; M's and B's sums
    const int row = tid / EACH_ROW;
    float sum = 0.f, m = 0.f, b = 0.f;
    for (int c = tid % EACH_ROW; c < V; c += EACH_ROW) {
      const float d = w.dr[(int64_t)row * V + c];
      sum = fmaf(d, v(row, c), sum);
      if (row < ch.len)
        static_cast<E *>(p.dv)[((ch.token + row) * p.H + head) * V + c] =
            from_f32<E>(f.beta[row] * d);
    }
    for (int j = tid % EACH_ROW; j < Q; j += EACH_ROW) {
      m += s.M[row * SIDE + j] + f.beta[row] * s.B[row * SIDE + j];
      m -= s.M[j * SIDE + row] + f.beta[j] * s.B[j * SIDE + row];
      b += s.B[row * SIDE + j];
    }
    sum = row_sum(sum);
    m = row_sum(m);
    b = row_sum(b);
    if (tid % EACH_ROW == 0) {
      dG[row] = m + qd[row] + f.beta[row] * kh[row];
      if (row < ch.len) p.dbeta[(ch.token + row) * p.H + head] = sum + kh[row] + b;
    }
    // <h, D>
    sum = 0.f;
    for (int x = tid; x < K * V; x += THREADS) sum = fmaf(w.h[x], w.D[x], sum);
    for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(~0u, sum, o);
    if (tid % 32 == 0) part[tid / 32] = sum;
    __syncthreads();
    if (tid < 32) {  // dG's sums from the end, two tokens a lane
      float kds[2] = {kD[tid], kD[tid + 32]};  // (zero past the end)
      float hD = 0.f, all = p.g_is_cumsum ? kds[0] + kds[1] : 0.f;
      for (int i = 0; i < THREADS / 32; ++i) hD += part[i];
      for (int o = 16; o > 0; o >>= 1) all += __shfl_xor_sync(~0u, all, o);
      float d[2];
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        const int i = tid + 32 * e;
        d[e] = i < ch.len ? dG[i] + (i == ch.len - 1 ? fmaf(keep, hD, all) : 0.f) : 0.f;
        if (p.g_is_cumsum) d[e] -= kds[e];
      }
      if (!p.g_is_cumsum) {
#pragma unroll
        for (int e = 0; e < 2; ++e)
#pragma unroll
          for (int o = 1; o < 32; o <<= 1) {
            const float x = __shfl_down_sync(~0u, d[e], o);
            if (tid + o < 32) d[e] += x;
          }
        d[0] += __shfl_sync(~0u, d[1], 0);
        delta_before(kds);
        d[0] += kds[0];
        d[1] += kds[1];
      }
#pragma unroll
      for (int e = 0; e < 2; ++e)
        if (tid + 32 * e < ch.len) p.dg[(ch.token + tid + 32 * e) * p.H + head] = d[e];
    }
    __syncthreads();
  }
  for (int x = tid; x < ch.len * K; x += THREADS) {
    const int64_t at = ((ch.token + x / K) * p.Hg + hk) * K + x % K;
    static_cast<E *>(p.dq)[at] = from_f32<E>(s.dq[x]);
    static_cast<E *>(p.dk)[at] = from_f32<E>(s.dk[x]);
  }
}

template <typename E>
cudaError_t launch(const DeltaBwdParams &p, cudaStream_t stream) {
  const dim3 walks((p.V + COLS - 1) / COLS, p.H, p.N);
  const int smem = Inputs::FLOATS * (int)sizeof(float);
  constexpr int PREPARE = (TILES + Q * SIDE) * (int)sizeof(float);
  cudaError_t e = cudaFuncSetAttribute(simt_inputs_kernel<E>,
                                       cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
  if (e == cudaSuccess)
    e = cudaFuncSetAttribute(simt_prepare_kernel<E>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                             PREPARE);
  if (e != cudaSuccess) return e;
  const dim3 all((unsigned)p.chunks, p.H);
  if (p.cu != nullptr) {
    e = launch_behind(simt_prepare_kernel<E>, all, THREADS, PREPARE, stream, p);
  } else {  // the call's first kernel
    simt_prepare_kernel<E><<<all, THREADS, PREPARE, stream>>>(p);
    e = cudaGetLastError();
  }
  if (e == cudaSuccess) e = launch_behind(simt_states_kernel<E>, walks, THREADS, 0, stream, p);
  if (e == cudaSuccess) e = launch_behind(simt_grads_kernel<E>, walks, THREADS, 0, stream, p);
  if (e != cudaSuccess) return e;
  return launch_behind(simt_inputs_kernel<E>, dim3((unsigned)p.chunks, p.Hg), THREADS, smem, stream, p);
}

}  // namespace

int64_t delta_bwd_simt_block(const DeltaBwdParams &p) {
  return (block_floats(p) * (int64_t)sizeof(float) + 255) / 256 * 256;
}

cudaError_t launch_delta_bwd_simt(const DeltaBwdParams &p, bool bf16, cudaStream_t stream) {
  return bf16 ? launch<__nv_bfloat16>(p, stream) : launch<float>(p, stream);
}

}  // namespace gdn
