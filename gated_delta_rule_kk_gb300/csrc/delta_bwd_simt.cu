// The gated delta rule's gradient over chunks on CUDA cores, in float32 throughout: every
// call that the tensor cores do not take (float32, odd head sizes, V > 128).  delta_bwd.h has
// the formulas.
//
// All products go through one tiled product of a block (64 x 64 outputs, 16 of them a thread,
// operands read through functions, so that gates, masks and transposes need no copies).
#include "delta_bwd.h"
#include "gdn_common.cuh"

namespace gdn {
namespace {

constexpr int Q = 64, THREADS = 256, COLS = 64;
constexpr int TILE = 16 * (Q + 4);  // floats of one operand's tile

// A chunk and head's floats: running log-gates and beta, T, P, n and dr [64][V], the state
// and its gradient [K][V].
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
};

int64_t block_floats(const DeltaBwdParams &p) {
  return 2 * Q + 2 * Q * Q + 2 * (int64_t)(Q + p.K) * p.V;
}

// out(i, j, sum_k a(i, k) b(k, j)) for i < M, j < N.  `tiles` is shared memory of 2 TILE
// floats.  Every operand is read before the first output of its 64 x 64 tile is written.
template <typename A, typename B, typename Out>
__device__ __forceinline__ void product(int M, int N, int K, float *tiles, A a, B b, Out out) {
  float *as = tiles, *bs = tiles + TILE;
  const int tid = threadIdx.x, ti = tid / 16 * 4, tj = tid % 16 * 4;
  for (int i0 = 0; i0 < M; i0 += 64)
    for (int j0 = 0; j0 < N; j0 += 64) {
      float acc[4][4] = {};
      for (int k0 = 0; k0 < K; k0 += 16) {
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const int x = tid + e * THREADS;
          const int ai = i0 + x / 16, ak = k0 + x % 16, bk = k0 + x / 64, bj = j0 + x % 64;
          as[x % 16 * 68 + x / 16] = ai < M && ak < K ? a(ai, ak) : 0.f;
          bs[x / 64 * 68 + x % 64] = bk < K && bj < N ? b(bk, bj) : 0.f;
        }
        __syncthreads();
#pragma unroll
        for (int k = 0; k < 16; ++k) {
          const float4 u = *reinterpret_cast<const float4 *>(as + k * 68 + ti);
          const float4 v = *reinterpret_cast<const float4 *>(bs + k * 68 + tj);
          const float x[4] = {u.x, u.y, u.z, u.w}, y[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
          for (int i = 0; i < 4; ++i)
#pragma unroll
            for (int j = 0; j < 4; ++j) acc[i][j] = fmaf(x[i], y[j], acc[i][j]);
        }
        __syncthreads();
      }
#pragma unroll
      for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int j = 0; j < 4; ++j)
          if (i0 + ti + i < M && j0 + tj + j < N) out(i0 + ti + i, j0 + tj + j, acc[i][j]);
    }
  __syncthreads();
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
    return i < len ? to_f32(at[i * stride + c]) : 0.f;
  }
};

// grid: chunks, heads.  G, beta, P, A and T = (I + A)^-1 by forward substitution, a column a
// thread (the columns of the identity, so that row i of T needs the rows before it).
template <typename E>
__global__ void __launch_bounds__(THREADS) simt_prepare_kernel(DeltaBwdParams p) {
  __shared__ __align__(16) float tiles[2 * TILE];
  __shared__ float A[Q][Q + 1], G[Q], beta[Q];
  const DeltaChunk ch = delta_chunk(p, blockIdx.x);
  const int head = blockIdx.y, hk = head / (p.H / p.Hg), tid = threadIdx.x;
  if (ch.len <= 0) return;
  if (!bounds_ok(ch.n < p.N && ch.token + ch.len <= (int64_t)p.B * p.T, p.err)) return;
  const Block w(p, blockIdx.x, head);
  if (tid < Q) {
    const int64_t at = (ch.token + min(tid, ch.len - 1)) * p.H + head;
    G[tid] = tid < ch.len || p.g_is_cumsum ? p.g[at] : 0.f;
    beta[tid] = tid < ch.len ? p.beta[at] : 0.f;
  }
  __syncthreads();
  if (tid == 0 && !p.g_is_cumsum)
    for (int i = 1; i < Q; ++i) G[i] += G[i - 1];
  __syncthreads();
  if (tid < Q) {
    w.G[tid] = G[tid];
    w.beta[tid] = beta[tid];
  }
  const Rows<E> q(p.q, ch.token, p.Hg, hk, p.K, ch.len), k(p.k, ch.token, p.Hg, hk, p.K, ch.len);
  auto kt = [&](int c, int j) { return k(j, c); };
  product(Q, Q, p.K, tiles, q, kt, [&](int i, int j, float s) {
    w.P[i * Q + j] = i >= j ? p.scale * s * expf(G[i] - G[j]) : 0.f;
  });
  product(Q, Q, p.K, tiles, k, kt, [&](int i, int j, float s) {
    A[i][j] = i > j ? beta[i] * s * expf(G[i] - G[j]) : 0.f;
  });
  if (tid < Q) {
    for (int i = 0; i < Q; ++i) {
      float s = i == tid ? 1.f : 0.f;
      for (int m = tid; m < i; ++m) s = fmaf(-A[i][m], w.T[m * Q + tid], s);
      w.T[i * Q + tid] = i >= tid ? s : 0.f;
    }
  }
}

// grid: 64 value columns, heads, sequences.  The states, forward.
template <typename E>
__global__ void __launch_bounds__(THREADS) simt_states_kernel(DeltaBwdParams p) {
  __shared__ __align__(16) float tiles[2 * TILE];
  const int v0 = blockIdx.x * COLS, nv = min(COLS, p.V - v0), head = blockIdx.y;
  const int hk = head / (p.H / p.Hg), K = p.K, V = p.V;
  int64_t first;
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
    product(Q, nv, K, tiles, k, [&](int i, int j) { return w.h[(int64_t)i * V + v0 + j]; },
            [&](int i, int j, float s) {
              w.n[(int64_t)i * V + v0 + j] = w.beta[i] * (v(i, v0 + j) - expf(w.G[i]) * s);
            });
    auto rows = [&](int i, int j) { return w.n[(int64_t)i * V + v0 + j]; };
    product(Q, nv, Q, tiles, [&](int i, int m) { return w.T[i * Q + m]; }, rows,
            [&](int i, int j, float s) { w.n[(int64_t)i * V + v0 + j] = s; });
    if (c + 1 == count) break;
    const Block next(p, first + c + 1, head);
    const float GL = w.G[ch.len - 1], keep = expf(GL);
    product(K, nv, ch.len, tiles, [&](int kc, int i) { return k(i, kc) * expf(GL - w.G[i]); }, rows,
            [&](int kc, int j, float s) {
              const int64_t at = (int64_t)kc * V + v0 + j;
              next.h[at] = fmaf(keep, w.h[at], s);
            });
  }
}

// grid: as simt_states_kernel.  The states' gradients, backward.
template <typename E>
__global__ void __launch_bounds__(THREADS) simt_grads_kernel(DeltaBwdParams p) {
  __shared__ __align__(16) float tiles[2 * TILE];
  const int v0 = blockIdx.x * COLS, nv = min(COLS, p.V - v0), head = blockIdx.y;
  const int hk = head / (p.H / p.Hg), K = p.K, V = p.V;
  int64_t first;
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
    const float GL = w.G[ch.len - 1], keep = expf(GL);
    product(Q, nv, Q, tiles, [&](int j, int i) { return w.P[i * Q + j]; },
            [&](int i, int j) { return go(i, v0 + j); },
            [&](int i, int j, float s) { w.dr[(int64_t)i * V + v0 + j] = s; });
    product(Q, nv, K, tiles, k, [&](int i, int j) { return w.D[(int64_t)i * V + v0 + j]; },
            [&](int i, int j, float s) {
              // (past the chunk's end k is zero and the gate may not be a sum)
              if (i < ch.len) w.dr[(int64_t)i * V + v0 + j] += expf(GL - w.G[i]) * s;
            });
    auto rows = [&](int i, int j) { return w.dr[(int64_t)i * V + v0 + j]; };
    product(Q, nv, Q, tiles, [&](int i, int m) { return w.T[m * Q + i]; }, rows,
            [&](int i, int j, float s) { w.dr[(int64_t)i * V + v0 + j] = s; });
    if (c == 0 && p.dh0 == nullptr) break;
    float *prev = c > 0 ? Block(p, first + c - 1, head).D : nullptr;
    product(K, nv, 2 * ch.len, tiles,
            [&](int kc, int i) {
              if (i < ch.len) return q(i, kc) * p.scale * expf(w.G[i]);
              i -= ch.len;
              return -k(i, kc) * w.beta[i] * expf(w.G[i]);
            },
            [&](int i, int j) { return i < ch.len ? go(i, v0 + j) : rows(i - ch.len, j); },
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
    dq = tiles + 2 * TILE;
    dk = dq + Q * KMAX;
    x = dk + Q * KMAX;
    P = x + Q * KMAX;
    A = P + Q * Q;
    M = A + Q * Q;
    B = M + Q * Q;
    sums = B + Q * Q;   // 8 x 64
  }
  static constexpr int FLOATS = 2 * TILE + 3 * Q * KMAX + 4 * Q * Q + 8 * Q;
};

// sum_c x[i][c] y(i, c) of every row, four threads a row, to out[i].
template <typename Y>
__device__ __forceinline__ void row_dots(const float *x, int K, Y y, float *out) {
  const int i = threadIdx.x / 4;
  float s = 0.f;
  for (int c = threadIdx.x % 4; c < K; c += 4) s = fmaf(x[i * K + c], y(i, c), s);
  s += __shfl_xor_sync(~0u, s, 1);
  s += __shfl_xor_sync(~0u, s, 2);
  if (threadIdx.x % 4 == 0) out[i] = s;
  __syncthreads();
}

// grid: chunks, key heads.  The gradients of a chunk's tokens; the value heads of a key head
// one after another, their dq and dk summed in shared memory.
template <typename E>
__global__ void __launch_bounds__(THREADS) simt_inputs_kernel(DeltaBwdParams p) {
  extern __shared__ __align__(16) float shared[];
  const Inputs s(shared);
  const DeltaChunk ch = delta_chunk(p, blockIdx.x);
  const int hk = blockIdx.y, rep = p.H / p.Hg, tid = threadIdx.x, K = p.K, V = p.V;
  if (ch.len <= 0) return;
  if (!bounds_ok(ch.n < p.N && ch.token + ch.len <= (int64_t)p.B * p.T, p.err)) return;
  const Rows<E> q(p.q, ch.token, p.Hg, hk, K, ch.len), k(p.k, ch.token, p.Hg, hk, K, ch.len);
  float *qd = s.sums, *kh = qd + Q, *kD = kh + Q, *rv = kD + Q, *dG = rv + Q, *part = dG + Q;
  for (int x = tid; x < Q * K; x += THREADS) s.dq[x] = s.dk[x] = 0.f;
  __syncthreads();
  for (int head = hk * rep; head < (hk + 1) * rep; ++head) {
    const Block w(p, blockIdx.x, head);
    const Rows<E> go(p.dout, ch.token, p.H, head, V, ch.len), v(p.v, ch.token, p.H, head, V, ch.len);
    const float GL = w.G[ch.len - 1], keep = expf(GL);
    auto kt = [&](int c, int j) { return k(j, c); };
    auto nt = [&](int c, int j) { return w.n[(int64_t)j * V + c]; };
    auto dr = [&](int i, int c) { return w.dr[(int64_t)i * V + c]; };
    auto ht = [&](int c, int kc) { return w.h[(int64_t)kc * V + c]; };
    product(Q, Q, K, s.tiles, q, kt, [&](int i, int j, float x) { s.P[i * Q + j] = x; });
    product(Q, Q, V, s.tiles, go, nt, [&](int i, int j, float x) {
      const float L = i >= j && i < ch.len ? p.scale * expf(w.G[i] - w.G[j]) : 0.f;
      s.M[i * Q + j] = L * x * s.P[i * Q + j];
      s.P[i * Q + j] = L * x;
    });
    product(Q, Q, K, s.tiles, k, kt, [&](int i, int j, float x) { s.A[i * Q + j] = x; });
    product(Q, Q, V, s.tiles, dr, nt, [&](int i, int j, float x) {
      const float L = i > j && i < ch.len ? expf(w.G[i] - w.G[j]) : 0.f;
      s.B[i * Q + j] = -L * x * s.A[i * Q + j];
      s.A[i * Q + j] = -L * x * w.beta[i];
    });
    product(Q, K, V, s.tiles, go, ht, [&](int i, int c, float x) {
      x *= p.scale * expf(w.G[i]);
      s.x[i * K + c] = x;
      s.dq[i * K + c] += x;
    });
    row_dots(s.x, K, q, qd);
    product(Q, K, V, s.tiles, dr, ht, [&](int i, int c, float x) {
      x *= -expf(w.G[i]);
      s.x[i * K + c] = x;
      s.dk[i * K + c] += w.beta[i] * x;
    });
    row_dots(s.x, K, k, kh);
    product(Q, K, V, s.tiles, [&](int i, int c) { return w.n[(int64_t)i * V + c]; },
            [&](int c, int kc) { return w.D[(int64_t)kc * V + c]; }, [&](int i, int c, float x) {
              x = i < ch.len ? x * expf(GL - w.G[i]) : 0.f;
              s.x[i * K + c] = x;
              s.dk[i * K + c] += x;
            });
    row_dots(s.x, K, k, kD);
    product(Q, K, Q, s.tiles, [&](int i, int j) { return s.P[i * Q + j]; }, k,
            [&](int i, int c, float x) { s.dq[i * K + c] += x; });
    product(Q, K, Q, s.tiles, [&](int j, int i) { return s.P[i * Q + j]; }, q,
            [&](int i, int c, float x) { s.dk[i * K + c] += x; });
    product(Q, K, Q, s.tiles, [&](int i, int j) { return s.A[i * Q + j] + s.A[j * Q + i]; }, k,
            [&](int i, int c, float x) { s.dk[i * K + c] += x; });
    // dr.v of every row, and dv
    const int row = tid / 4;
    float sum = 0.f;
    for (int c = tid % 4; c < V; c += 4) {
      const float d = w.dr[(int64_t)row * V + c];
      sum = fmaf(d, v(row, c), sum);
      if (row < ch.len)
        static_cast<E *>(p.dv)[((ch.token + row) * p.H + head) * V + c] =
            from_f32<E>(w.beta[row] * d);
    }
    sum += __shfl_xor_sync(~0u, sum, 1);
    sum += __shfl_xor_sync(~0u, sum, 2);
    if (tid % 4 == 0) rv[row] = sum;
    // <h, D>
    sum = 0.f;
    for (int x = tid; x < K * V; x += THREADS) sum = fmaf(w.h[x], w.D[x], sum);
    for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(~0u, sum, o);
    if (tid % 32 == 0) part[tid / 32] = sum;
    __syncthreads();
    if (tid < Q) {
      float m = 0.f, b = 0.f;
      for (int j = 0; j < Q; ++j) {
        m += s.M[tid * Q + j] + w.beta[tid] * s.B[tid * Q + j];
        m -= s.M[j * Q + tid] + w.beta[j] * s.B[j * Q + tid];
        b += s.B[tid * Q + j];
      }
      dG[tid] = m + qd[tid] + w.beta[tid] * kh[tid] - kD[tid];
      if (tid < ch.len) p.dbeta[(ch.token + tid) * p.H + head] = rv[tid] + kh[tid] + b;
    }
    __syncthreads();
    if (tid == 0) {
      float hD = 0.f, all = 0.f;
      for (int i = 0; i < THREADS / 32; ++i) hD += part[i];
      for (int i = 0; i < ch.len; ++i) all += kD[i];
      dG[ch.len - 1] += fmaf(keep, hD, all);
      float run = 0.f;
      for (int i = ch.len - 1; i >= 0; --i) {
        run = p.g_is_cumsum ? dG[i] : run + dG[i];
        p.dg[(ch.token + i) * p.H + head] = run;
      }
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
  const cudaError_t e = cudaFuncSetAttribute(simt_inputs_kernel<E>,
                                             cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
  if (e != cudaSuccess) return e;
  simt_prepare_kernel<E><<<dim3((unsigned)p.chunks, p.H), THREADS, 0, stream>>>(p);
  simt_states_kernel<E><<<walks, THREADS, 0, stream>>>(p);
  simt_grads_kernel<E><<<walks, THREADS, 0, stream>>>(p);
  simt_inputs_kernel<E><<<dim3((unsigned)p.chunks, p.Hg), THREADS, smem, stream>>>(p);
  return cudaGetLastError();
}

}  // namespace

int64_t delta_bwd_simt_block(const DeltaBwdParams &p) {
  return (block_floats(p) * (int64_t)sizeof(float) + 255) / 256 * 256;
}

cudaError_t launch_delta_bwd_simt(const DeltaBwdParams &p, bool bf16, cudaStream_t stream) {
  return bf16 ? launch<__nv_bfloat16>(p, stream) : launch<float>(p, stream);
}

}  // namespace gdn
