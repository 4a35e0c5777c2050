// The gated delta rule's gradient over chunks on the tensor cores: bfloat16 inputs, K and V
// multiples of 8, K <= 128, V <= 128.  delta_bwd.h has the formulas.
//
// Every product is of 64 x 64 x 32 .. 64 x 128 x 128 and stands between element-wise gates,
// masks and sums, so accumulators stay in registers (warp-level matrix instructions) instead
// of passing through tensor memory between each two of them.  q, k, v and do are bfloat16 and
// exact; what is float32 (T, P, the states h and their gradients D, the corrected values n and
// dr) enters as a pair of bfloat16 pieces, hi + lo, with the products hi hi + hi lo + lo hi:
// off by 2^-17 of each value at most, so that the float32 results (dg, dbeta, dh0) are not
// bound by bfloat16.  Accumulation is float32.
//
// Matrices lie in shared memory as rows of 64, 128 or 256 bytes whose 16-byte pieces are
// exchanged by row (`at`), so that matrix loads touch every bank once; the workspace holds
// the same images, so that the next kernel fetches them by straight copies.
#include <algorithm>

#include "delta_bwd.h"
#include "gdn_common.cuh"
#include "ptx.cuh"

namespace gdn {
namespace {

using bf16 = __nv_bfloat16;

constexpr int Q = 64;    // tokens of a chunk
constexpr int VT = 32;   // value columns of a tile

// Place of (row, col) in an image with rows of COLS elements.
template <int COLS>
__device__ __forceinline__ int at(int row, int col) {
  const int turn = COLS == 32 ? (row >> 1) & 3 : row & 7;
  return row * COLS + (((col >> 3) ^ turn) << 3) + (col & 7);
}

// Fragments of m16n8k16.  A from rows [m][k] or (lda_t) from [k][m]; B, two tiles of eight
// columns, from [n][k] or (ldb_t) from [k][n].
template <int COLS>
__device__ __forceinline__ void lda(uint32_t (&a)[4], const bf16 *s, int m0, int k0) {
  const int l = threadIdx.x & 31;
  ptx::ldmatrix_x4(s + at<COLS>(m0 + (l & 15), k0 + (l >> 4) * 8), a[0], a[1], a[2], a[3]);
}
template <int COLS>
__device__ __forceinline__ void lda_t(uint32_t (&a)[4], const bf16 *s, int m0, int k0) {
  const int l = threadIdx.x & 31;
  ptx::ldmatrix_x4_trans(s + at<COLS>(k0 + (l & 7) + (l >> 4) * 8, m0 + ((l >> 3) & 1) * 8), a[0],
                         a[1], a[2], a[3]);
}
template <int COLS>
__device__ __forceinline__ void ldb(uint32_t (&b)[4], const bf16 *s, int n0, int k0) {
  const int l = threadIdx.x & 31;
  ptx::ldmatrix_x4(s + at<COLS>(n0 + (l & 7) + (l >> 4) * 8, k0 + ((l >> 3) & 1) * 8), b[0], b[1],
                   b[2], b[3]);
}
template <int COLS>
__device__ __forceinline__ void ldb_t(uint32_t (&b)[4], const bf16 *s, int n0, int k0) {
  const int l = threadIdx.x & 31;
  ptx::ldmatrix_x4_trans(s + at<COLS>(k0 + (l & 7) + ((l >> 3) & 1) * 8, n0 + (l >> 4) * 8), b[0],
                         b[1], b[2], b[3]);
}

// c (16 x 16) += a b
__device__ __forceinline__ void mma2(float (*c)[4], const uint32_t (&a)[4], const uint32_t (&b)[4]) {
  ptx::mma_16816_bf16(c[0], a, b[0], b[1]);
  ptx::mma_16816_bf16(c[1], a, b[2], b[3]);
}

// x and y (neighbouring columns) as pieces to images hi and lo.
__device__ __forceinline__ void put_pair(bf16 *hi, bf16 *lo, int place, float x, float y) {
  const __nv_bfloat162 h = __floats2bfloat162_rn(x, y);
  const float2 f = __bfloat1622float2(h);
  *reinterpret_cast<__nv_bfloat162 *>(hi + place) = h;
  *reinterpret_cast<__nv_bfloat162 *>(lo + place) = __floats2bfloat162_rn(x - f.x, y - f.y);
}

__device__ __forceinline__ float2 get_pair(const bf16 *s, int place) {
  return __bfloat1622float2(*reinterpret_cast<const __nv_bfloat162 *>(s + place));
}

// A chunk and head in the workspace (bytes; KP = K rounded up to 64 or 128): gates and beta,
// then images, each hi then lo: T, P; by value tiles n, dr [64][32], h, D [KP][32].
template <int KP>
struct Block {
  static constexpr int SC = 2 * Q * 4, SQUARE = 2 * Q * Q * 2, ROWS = 2 * Q * VT * 2,
                       STATE = 2 * KP * VT * 2;
  unsigned char *base;
  int tiles;
  __device__ Block(const DeltaBwdParams &p, int64_t chunk, int head)
      : base(p.blocks + (chunk * p.H + head) * p.block), tiles((p.V + VT - 1) / VT) {}
  __device__ float *sc() const { return reinterpret_cast<float *>(base); }
  __device__ unsigned char *T() const { return base + SC; }
  __device__ unsigned char *P() const { return base + SC + SQUARE; }
  __device__ unsigned char *n(int v) const { return base + SC + 2 * SQUARE + v * ROWS; }
  __device__ unsigned char *dr(int v) const { return n(tiles) + v * ROWS; }
  __device__ unsigned char *h(int v) const { return dr(tiles) + v * STATE; }
  __device__ unsigned char *D(int v) const { return h(tiles) + v * STATE; }
  static int64_t bytes(int tiles) {
    return SC + 2 * SQUARE + (int64_t)tiles * 2 * (ROWS + STATE);
  }
};

// Straight copies between shared memory and the workspace, by all threads.
template <int THREADS>
__device__ __forceinline__ void fetch(void *to, const void *from, int bytes) {
  for (int i = threadIdx.x * 16; i < bytes; i += THREADS * 16)
    ptx::cp_async16(static_cast<unsigned char *>(to) + i,
                    static_cast<const unsigned char *>(from) + i, true);
}
template <int THREADS>
__device__ __forceinline__ void keep(void *to, const void *from, int bytes) {
  for (int i = threadIdx.x * 16; i < bytes; i += THREADS * 16)
    *reinterpret_cast<uint4 *>(static_cast<unsigned char *>(to) + i) =
        *reinterpret_cast<const uint4 *>(static_cast<const unsigned char *>(from) + i);
}

// Columns c0 .. c0 + COLS - 1 of a chunk's rows of a tensor [.., heads, D] as an image; zero
// past the chunk's end and past D.
template <int COLS, int THREADS>
__device__ __forceinline__ void fetch_rows(bf16 *to, const void *tensor, const DeltaChunk &ch,
                                           int heads, int head, int D, int c0) {
  const bf16 *from = static_cast<const bf16 *>(tensor) + (ch.token * heads + head) * D;
  const int64_t stride = (int64_t)heads * D;
  for (int i = threadIdx.x; i < Q * COLS / 8; i += THREADS) {
    const int row = i / (COLS / 8), col = i % (COLS / 8) * 8;
    const bool ok = row < ch.len && c0 + col < D;
    ptx::cp_async16(to + at<COLS>(row, col), ok ? from + row * stride + c0 + col : from, ok);
  }
}

// ---------------------------------------------------------------- T and P

// grid: chunks, heads.  Running log-gates, P and T = (I + A)^-1.  [q; k] k^T on the tensor
// cores; the inverse in float32 on CUDA cores: the four 16 x 16 blocks on the diagonal by
// forward substitution, a column a thread, then the blocks below it, a diagonal at a time,
// T_(b+d, b) = -T_(b+d, b+d) sum_m A_(b+d, m) T_(m, b).
constexpr int PREP = 256;
template <int KP>
struct PrepareShared {
  static constexpr int IMAGES = 2 * Block<KP>::SQUARE;  // q and k, then T and P
  static constexpr int BYTES = IMAGES + (2 * Q * (Q + 1) + 3 * 16 * 17 + 2 * Q) * 4;
};

template <int KP>
__global__ void __launch_bounds__(PREP, 3) tc_prepare_kernel(DeltaBwdParams p) {
  extern __shared__ __align__(128) unsigned char shared[];
  bf16 *q = reinterpret_cast<bf16 *>(shared), *k = q + Q * KP;
  float(*A)[Q + 1] = reinterpret_cast<float(*)[Q + 1]>(shared + PrepareShared<KP>::IMAGES);
  float(*T)[Q + 1] = A + Q;
  float(*X)[16][17] = reinterpret_cast<float(*)[16][17]>(T + Q);
  float *G = reinterpret_cast<float *>(X + 3), *beta = G + Q;
  const DeltaChunk ch = delta_chunk(p, blockIdx.x);
  const int head = blockIdx.y, hk = head / (p.H / p.Hg);
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  if (ch.len <= 0) return;
  if (!bounds_ok(ch.n < p.N && ch.token + ch.len <= (int64_t)p.B * p.T && blockIdx.x < p.chunks,
                 p.err))
    return;
  const Block<KP> w(p, blockIdx.x, head);
  fetch_rows<KP, PREP>(q, p.q, ch, p.Hg, hk, p.K, 0);
  fetch_rows<KP, PREP>(k, p.k, ch, p.Hg, hk, p.K, 0);
  ptx::cp_async_commit();
  if (warp == 0) {
    float g[2];
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      const int i = lane + 32 * e;
      const int64_t where = (ch.token + min(i, ch.len - 1)) * p.H + head;
      g[e] = i < ch.len || p.g_is_cumsum ? p.g[where] : 0.f;
      beta[i] = i < ch.len ? p.beta[where] : 0.f;
    }
    if (!p.g_is_cumsum) {
#pragma unroll
      for (int e = 0; e < 2; ++e)
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
          const float v = __shfl_up_sync(~0u, g[e], o);
          if (lane >= o) g[e] += v;
        }
      g[1] += __shfl_sync(~0u, g[0], 31);
    }
    G[lane] = g[0];
    G[lane + 32] = g[1];
  }
  ptx::cp_async_wait<0>();
  __syncthreads();
  if (tid < Q) {
    w.sc()[tid] = G[tid];
    w.sc()[Q + tid] = beta[tid];
  }
  const int wm = warp & 3, g = lane >> 2, t = lane & 3;
  const bool of_q = warp < 4;
  float s[8][4] = {};
  for (int kk = 0; kk < KP; kk += 16) {
    uint32_t a[4], b[4];
    lda<KP>(a, of_q ? q : k, 16 * wm, kk);
#pragma unroll
    for (int j = 0; j < 4; ++j)
      if (j <= wm) {
        ldb<KP>(b, k, 16 * j, kk);
        mma2(s + 2 * j, a, b);
      }
  }
  __syncthreads();  // q and k have been read
  bf16 *Th = reinterpret_cast<bf16 *>(shared), *Tl = Th + Q * Q, *Ph = Tl + Q * Q, *Pl = Ph + Q * Q;
#pragma unroll
  for (int j = 0; j < 8; ++j)
#pragma unroll
    for (int r = 0; r < 2; ++r) {
      const int row = 16 * wm + g + 8 * r, col = 8 * j + 2 * t;
      float v[2];
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        const bool in = of_q ? row >= col + e : row > col + e;
        v[e] = in ? (of_q ? p.scale : beta[row]) * s[j][2 * r + e] * __expf(G[row] - G[col + e]) : 0.f;
      }
      if (of_q) {
        put_pair(Ph, Pl, at<64>(row, col), v[0], v[1]);
      } else {
        A[row][col] = v[0];
        A[row][col + 1] = v[1];
      }
    }
  __syncthreads();
  if (tid < Q) {
    const int b = tid / 16 * 16, j = tid % 16;
    float x[16];
#pragma unroll
    for (int i = 0; i < 16; ++i) {
      x[i] = i == j ? 1.f : 0.f;
#pragma unroll
      for (int m = 0; m < i; ++m) x[i] = fmaf(-A[b + i][b + m], x[m], x[i]);
      T[b + i][b + j] = x[i];
    }
  }
  __syncthreads();
  const int bi = tid / 16, bj = tid % 16;
#pragma unroll
  for (int d = 1; d < 4; ++d) {
#pragma unroll
    for (int b = 0; b + d < 4; ++b) {
      float x = 0.f;
#pragma unroll
      for (int m = 0; m < 16 * d; ++m) x = fmaf(A[16 * (b + d) + bi][16 * b + m], T[16 * b + m][16 * b + bj], x);
      X[b][bi][bj] = x;
    }
    __syncthreads();
#pragma unroll
    for (int b = 0; b + d < 4; ++b) {
      float x = 0.f;
#pragma unroll
      for (int m = 0; m < 16; ++m) x = fmaf(T[16 * (b + d) + bi][16 * (b + d) + m], X[b][m][bj], x);
      T[16 * (b + d) + bi][16 * b + bj] = -x;
    }
    __syncthreads();
  }
  for (int i = tid; i < Q * Q / 2; i += PREP) {
    const int row = i / 32, col = i % 32 * 2;
    put_pair(Th, Tl, at<64>(row, col), row >= col ? T[row][col] : 0.f,
             row >= col + 1 ? T[row][col + 1] : 0.f);
  }
  __syncthreads();
  keep<PREP>(w.T(), shared, 2 * Block<KP>::SQUARE);
}

// ---------------------------------------------------------------- the states, both ways

constexpr int WALK = 256;

// A walk's warp: rows 16 wm, columns 16 wn of the 64 x 32 products; rows 16 sm, columns sn ..
// of the state's tile [KP][32].
template <int KP>
struct WalkWarp {
  static constexpr int PARTS = WALK / 32 / (KP / 16), NT = 4 / PARTS;  // tiles of 8 columns
  int lane, wm, wn, g, t, sm, sn;
  __device__ WalkWarp() {
    const int warp = threadIdx.x >> 5;
    lane = threadIdx.x & 31;
    wm = warp & 3;
    wn = warp >> 2;
    g = lane >> 2;
    t = lane & 3;
    sm = warp % (KP / 16) * 16;
    sn = warp / (KP / 16) * 8 * NT;
  }
  __device__ int row(int r) const { return 16 * wm + g + 8 * r; }
  __device__ int col(int j) const { return 16 * wn + 8 * j + 2 * t; }
  __device__ int srow(int r) const { return sm + g + 8 * r; }
  __device__ int scol(int j) const { return sn + 8 * j + 2 * t; }
};

// Element (c, j) of a sequence and head's state tensor.
__device__ __forceinline__ int64_t state_at(const DeltaBwdParams &p, int n, int head, int c, int j) {
  return ((int64_t)n * p.H + head) * p.K * p.V +
         (p.v_first ? (int64_t)j * p.K + c : (int64_t)c * p.V + j);
}

template <int KP>
__device__ __forceinline__ void load_state(const DeltaBwdParams &p, const WalkWarp<KP> &m,
                                           const float *from, int n, int head, int v0,
                                           float (*s)[4]) {
#pragma unroll
  for (int j = 0; j < WalkWarp<KP>::NT; ++j)
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const int c = m.srow(e >> 1), v = v0 + m.scol(j) + (e & 1);
      s[j][e] = from && c < p.K && v < p.V ? from[state_at(p, n, head, c, v)] : 0.f;
    }
}

template <int KP>
__device__ __forceinline__ void put_state(const WalkWarp<KP> &m, bf16 *hi, const float (*s)[4]) {
#pragma unroll
  for (int j = 0; j < WalkWarp<KP>::NT; ++j)
#pragma unroll
    for (int r = 0; r < 2; ++r)
      put_pair(hi, hi + KP * VT, at<32>(m.srow(r), m.scol(j)), s[j][2 * r], s[j][2 * r + 1]);
}

// s += a^T (b_hi + b_lo) over 64 tokens: a [token][KP], b [token][32].
template <int KP>
__device__ __forceinline__ void add_outer(const WalkWarp<KP> &m, float (*s)[4], const bf16 *a,
                                          const bf16 *b) {
#pragma unroll
  for (int kk = 0; kk < Q; kk += 16) {
    uint32_t x[4], y[4];
    lda_t<KP>(x, a, m.sm, kk);
#pragma unroll
    for (int j = 0; j < WalkWarp<KP>::NT; j += 2) {
      ldb_t<32>(y, b, m.sn + 8 * j, kk);
      mma2(s + j, x, y);
      ldb_t<32>(y, b + Q * VT, m.sn + 8 * j, kk);
      mma2(s + j, x, y);
    }
  }
}

// c (16 x 16) = k (s_hi + s_lo): k [token][KP], s [KP][32].
template <int KP>
__device__ __forceinline__ void times_state(const WalkWarp<KP> &m, float (*c)[4], const bf16 *k,
                                            const bf16 *s) {
  float lo[2][4] = {};
#pragma unroll
  for (int kk = 0; kk < KP; kk += 16) {
    uint32_t a[4], b[4];
    lda<KP>(a, k, 16 * m.wm, kk);
    ldb_t<32>(b, s, 16 * m.wn, kk);
    mma2(c, a, b);
    ldb_t<32>(b, s + KP * VT, 16 * m.wn, kk);
    mma2(lo, a, b);
  }
#pragma unroll
  for (int j = 0; j < 2; ++j)
#pragma unroll
    for (int e = 0; e < 4; ++e) c[j][e] += lo[j][e];
}

// c (16 x 16) = T x or (BACK) T^T x, both as pieces; T's upper triangle is zero.
template <bool BACK>
__device__ __forceinline__ void times_T(int wm, int wn, float (*c)[4], const bf16 *T, const bf16 *x) {
  float lo[2][4] = {};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    if (BACK ? i < wm : i > wm) continue;
    uint32_t a[4], b[4], l[4];
    if (BACK)
      lda_t<64>(a, T, 16 * wm, 16 * i);
    else
      lda<64>(a, T, 16 * wm, 16 * i);
    ldb_t<32>(b, x, 16 * wn, 16 * i);
    mma2(c, a, b);
    ldb_t<32>(l, x + Q * VT, 16 * wn, 16 * i);
    mma2(lo, a, l);
    if (BACK)
      lda_t<64>(a, T + Q * Q, 16 * wm, 16 * i);
    else
      lda<64>(a, T + Q * Q, 16 * wm, 16 * i);
    mma2(lo, a, b);
  }
#pragma unroll
  for (int j = 0; j < 2; ++j)
#pragma unroll
    for (int e = 0; e < 4; ++e) c[j][e] += lo[j][e];
}

// Shared memory of the forward walk.
template <int KP>
struct StatesShared {
  static constexpr int K_ = Q * KP * 2, T_ = Block<KP>::SQUARE, V_ = Q * VT * 2, SC_ = Block<KP>::SC;
  static constexpr int STAGE = K_ + T_ + V_ + SC_;
  static constexpr int H = 2 * STAGE, R = H + Block<KP>::STATE, N = R + Block<KP>::ROWS;
  static constexpr int BYTES = N + Block<KP>::ROWS;
};

// grid: value tiles, heads, sequences.  The state's tile stays in registers; its pieces go to
// shared memory for k h and, a chunk each, to the workspace.
template <int KP>
__global__ void __launch_bounds__(WALK, 2) tc_states_kernel(DeltaBwdParams p) {
  using S = StatesShared<KP>;
  extern __shared__ __align__(128) unsigned char shared[];
  const int vt = blockIdx.x, v0 = vt * VT, head = blockIdx.y, n = blockIdx.z;
  const int hk = head / (p.H / p.Hg);
  const WalkWarp<KP> m;
  int64_t first;
  if (!delta_good(p)) return;
  const int count = delta_chunks(p, n, &first);
  if (count == 0) return;
  if (!bounds_ok(v0 < p.V && head < p.H && n < p.N && first + count <= p.chunks, p.err)) return;
  bf16 *h = reinterpret_cast<bf16 *>(shared + S::H);
  bf16 *r = reinterpret_cast<bf16 *>(shared + S::R), *nt = reinterpret_cast<bf16 *>(shared + S::N);
  auto load = [&](int c) {
    unsigned char *to = shared + (c & 1) * S::STAGE;
    const DeltaChunk ch = delta_chunk(p, first + c);
    const Block<KP> w(p, first + c, head);
    fetch_rows<KP, WALK>(reinterpret_cast<bf16 *>(to), p.k, ch, p.Hg, hk, p.K, 0);
    fetch<WALK>(to + S::K_, w.T(), S::T_);
    fetch_rows<32, WALK>(reinterpret_cast<bf16 *>(to + S::K_ + S::T_), p.v, ch, p.H, head, p.V, v0);
    fetch<WALK>(to + S::K_ + S::T_ + S::V_, w.sc(), S::SC_);
    ptx::cp_async_commit();
  };
  load(0);
  float s[WalkWarp<KP>::NT][4];
  load_state<KP>(p, m, p.h0, n, head, v0, s);
  put_state<KP>(m, h, s);
  ptx::cp_async_wait<0>();
  __syncthreads();
  for (int c = 0; c < count; ++c) {
    const unsigned char *in = shared + (c & 1) * S::STAGE;
    const bf16 *k = reinterpret_cast<const bf16 *>(in);
    const bf16 *T = reinterpret_cast<const bf16 *>(in + S::K_);
    const bf16 *v = reinterpret_cast<const bf16 *>(in + S::K_ + S::T_);
    const float *G = reinterpret_cast<const float *>(in + S::K_ + S::T_ + S::V_), *beta = G + Q;
    const Block<KP> w(p, first + c, head);
    if (c + 1 < count) load(c + 1);
    keep<WALK>(w.h(vt), h, Block<KP>::STATE);
    float x[2][4] = {};
    times_state<KP>(m, x, k, h);
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      const int i = m.row(e);
      const float eG = __expf(G[i]), b = beta[i];
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        const int place = at<32>(i, m.col(j));
        const float2 u = get_pair(v, place);
        put_pair(r, r + Q * VT, place, b * fmaf(-eG, x[j][2 * e], u.x),
                 b * fmaf(-eG, x[j][2 * e + 1], u.y));
      }
    }
    __syncthreads();
    float y[2][4] = {};
    times_T<false>(m.wm, m.wn, y, T, r);
    __syncthreads();  // r has been read
    const float GL = G[Q - 1];
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      const int i = m.row(e);
      const float f = __expf(GL - G[i]);
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        const int place = at<32>(i, m.col(j));
        put_pair(r, r + Q * VT, place, y[j][2 * e], y[j][2 * e + 1]);
        put_pair(nt, nt + Q * VT, place, f * y[j][2 * e], f * y[j][2 * e + 1]);
      }
    }
    __syncthreads();
    keep<WALK>(w.n(vt), r, Block<KP>::ROWS);
    if (c + 1 == count) break;
    const float eL = __expf(GL);
#pragma unroll
    for (int j = 0; j < WalkWarp<KP>::NT; ++j)
#pragma unroll
      for (int e = 0; e < 4; ++e) s[j][e] *= eL;
    add_outer<KP>(m, s, k, nt);
    put_state<KP>(m, h, s);
    ptx::cp_async_wait<0>();
    __syncthreads();
  }
}

// Shared memory of the backward walk.
template <int KP>
struct GradsShared {
  static constexpr int K_ = Q * KP * 2, TP_ = 2 * Block<KP>::SQUARE, V_ = Q * VT * 2,
                       SC_ = Block<KP>::SC;
  static constexpr int STAGE = 2 * K_ + TP_ + V_ + SC_;
  static constexpr int D = 2 * STAGE, R = D + Block<KP>::STATE, O = R + Block<KP>::ROWS,
                       B = O + Block<KP>::ROWS;
  static constexpr int BYTES = B + Block<KP>::ROWS;
};

// grid: as tc_states_kernel, from the last chunk to the first.
template <int KP>
__global__ void __launch_bounds__(WALK, 1) tc_grads_kernel(DeltaBwdParams p) {
  using S = GradsShared<KP>;
  extern __shared__ __align__(128) unsigned char shared[];
  const int vt = blockIdx.x, v0 = vt * VT, head = blockIdx.y, n = blockIdx.z;
  const int hk = head / (p.H / p.Hg);
  const WalkWarp<KP> m;
  int64_t first;
  if (!delta_good(p)) return;
  const int count = delta_chunks(p, n, &first);
  if (!bounds_ok(v0 < p.V && head < p.H && n < p.N && first + count <= p.chunks, p.err)) return;
  bf16 *D = reinterpret_cast<bf16 *>(shared + S::D), *r = reinterpret_cast<bf16 *>(shared + S::R);
  bf16 *od = reinterpret_cast<bf16 *>(shared + S::O), *rd = reinterpret_cast<bf16 *>(shared + S::B);
  auto load = [&](int c) {
    unsigned char *to = shared + (c & 1) * S::STAGE;
    const DeltaChunk ch = delta_chunk(p, first + c);
    const Block<KP> w(p, first + c, head);
    fetch_rows<KP, WALK>(reinterpret_cast<bf16 *>(to), p.k, ch, p.Hg, hk, p.K, 0);
    fetch_rows<KP, WALK>(reinterpret_cast<bf16 *>(to + S::K_), p.q, ch, p.Hg, hk, p.K, 0);
    fetch<WALK>(to + 2 * S::K_, w.T(), S::TP_);  // P lies behind T
    fetch_rows<32, WALK>(reinterpret_cast<bf16 *>(to + 2 * S::K_ + S::TP_), p.dout, ch, p.H, head,
                         p.V, v0);
    fetch<WALK>(to + 2 * S::K_ + S::TP_ + S::V_, w.sc(), S::SC_);
    ptx::cp_async_commit();
  };
  if (count > 0) load(count - 1);
  float s[WalkWarp<KP>::NT][4];
  load_state<KP>(p, m, p.dht, n, head, v0, s);
  put_state<KP>(m, D, s);
  ptx::cp_async_wait<0>();
  __syncthreads();
  for (int c = count - 1; c >= 0; --c) {
    const unsigned char *in = shared + (c & 1) * S::STAGE;
    const bf16 *k = reinterpret_cast<const bf16 *>(in);
    const bf16 *q = reinterpret_cast<const bf16 *>(in + S::K_);
    const bf16 *T = reinterpret_cast<const bf16 *>(in + 2 * S::K_), *P = T + 2 * Q * Q;
    const bf16 *go = reinterpret_cast<const bf16 *>(in + 2 * S::K_ + S::TP_);
    const float *G = reinterpret_cast<const float *>(in + 2 * S::K_ + S::TP_ + S::V_), *beta = G + Q;
    const Block<KP> w(p, first + c, head);
    if (c > 0) load(c - 1);
    keep<WALK>(w.D(vt), D, Block<KP>::STATE);
    float x[2][4] = {}, y[2][4] = {};
    times_state<KP>(m, x, k, D);
#pragma unroll
    for (int i = 0; i < 4; ++i) {  // P^T do
      if (i < m.wm) continue;
      uint32_t a[4], b[4];
      ldb_t<32>(b, go, 16 * m.wn, 16 * i);
      lda_t<64>(a, P, 16 * m.wm, 16 * i);
      mma2(y, a, b);
      lda_t<64>(a, P + Q * Q, 16 * m.wm, 16 * i);
      mma2(y, a, b);
    }
    const float GL = G[Q - 1];
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      const int i = m.row(e);
      const float f = __expf(GL - G[i]), o = p.scale * __expf(G[i]);
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        const int place = at<32>(i, m.col(j));
        put_pair(r, r + Q * VT, place, fmaf(f, x[j][2 * e], y[j][2 * e]),
                 fmaf(f, x[j][2 * e + 1], y[j][2 * e + 1]));
        const float2 d = get_pair(go, place);
        put_pair(od, od + Q * VT, place, o * d.x, o * d.y);
      }
    }
    __syncthreads();
    float z[2][4] = {};
    times_T<true>(m.wm, m.wn, z, T, r);
    __syncthreads();  // dn has been read
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      const int i = m.row(e);
      const float f = -beta[i] * __expf(G[i]);
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        const int place = at<32>(i, m.col(j));
        put_pair(r, r + Q * VT, place, z[j][2 * e], z[j][2 * e + 1]);
        put_pair(rd, rd + Q * VT, place, f * z[j][2 * e], f * z[j][2 * e + 1]);
      }
    }
    __syncthreads();
    keep<WALK>(w.dr(vt), r, Block<KP>::ROWS);
    const float eL = __expf(GL);
#pragma unroll
    for (int j = 0; j < WalkWarp<KP>::NT; ++j)
#pragma unroll
      for (int e = 0; e < 4; ++e) s[j][e] *= eL;
    add_outer<KP>(m, s, q, od);
    add_outer<KP>(m, s, k, rd);
    if (c == 0) break;
    put_state<KP>(m, D, s);
    ptx::cp_async_wait<0>();
    __syncthreads();
  }
  if (p.dh0 == nullptr) return;
#pragma unroll
  for (int j = 0; j < WalkWarp<KP>::NT; ++j)
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const int c = m.srow(e >> 1), v = v0 + m.scol(j) + (e & 1);
      if (c < p.K && v < p.V) p.dh0[state_at(p, n, head, c, v)] = s[j][e];
    }
}

// ---------------------------------------------------------------- the inputs' gradients

constexpr int IN = 512;

template <int KP>
struct InputsShared {
  static constexpr int K_ = Q * KP * 2, V_ = Q * VT * 2;
  static constexpr int ROWS = Block<KP>::ROWS, STATE = Block<KP>::STATE;
  // a value tile: do, v, dr, n, h, D; the second one's place then holds dP L and dA L beta
  static constexpr int STAGE = std::max(2 * V_ + 2 * ROWS + 2 * STATE, 2 * Block<KP>::SQUARE);
  static constexpr int STAGES = 2 * K_, SUMS = STAGES + 2 * STAGE;
  static constexpr int SUM_FLOATS = 27 * Q + 16;
  static constexpr int TOTALS = SUMS + SUM_FLOATS * 4;
  static constexpr int bytes(bool grouped) { return TOTALS + (grouped ? 2 * Q * KP * 4 : 0); }
};

// Sums of both rows of a thread's fragment over the row's four lanes.
__device__ __forceinline__ void put_rows(float *to, int row, int t, float a, float b) {
  a += __shfl_xor_sync(~0u, a, 1);
  b += __shfl_xor_sync(~0u, b, 1);
  a += __shfl_xor_sync(~0u, a, 2);
  b += __shfl_xor_sync(~0u, b, 2);
  if (t == 0) {
    to[row] = a;
    to[row + 8] = b;
  }
}

// grid: chunks, key heads.  16 warps: rows 16 wm, a quarter wn of the columns.  The value
// tiles stream through two stages; do h^T, dr h^T, n D^T, do n^T and dr n^T accumulate over
// them in registers (64 a thread).  The value heads of a key head follow one another, their
// dq and dk summed in shared memory (GROUPED).
template <int KP, bool GROUPED>
__global__ void __launch_bounds__(IN, 1) tc_inputs_kernel(DeltaBwdParams p) {
  using S = InputsShared<KP>;
  constexpr int NT = KP / 32;  // tiles of 8 columns of a warp's part of [64][KP]
  extern __shared__ __align__(128) unsigned char shared[];
  bf16 *q = reinterpret_cast<bf16 *>(shared), *k = q + Q * KP;
  float *sums = reinterpret_cast<float *>(shared + S::SUMS);
  // by quarters: q.dq_h, k.dk_h / beta, k.dk_s, rows of M, rows of B; columns of M by wm
  float *qd = sums, *kh = qd + 4 * Q, *kD = kh + 4 * Q, *rM = kD + 4 * Q, *rB = rM + 4 * Q;
  float *cM = rB + 4 * Q, *rv = cM + 4 * Q, *sc = rv + Q, *hD = sc + 2 * Q;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int wm = warp & 3, wn = warp >> 2, g = lane >> 2, t = lane & 3;
  const DeltaChunk ch = delta_chunk(p, blockIdx.x);
  const int hk = blockIdx.y, rep = p.H / p.Hg, tiles = (p.V + VT - 1) / VT;
  if (ch.len <= 0) return;
  if (!bounds_ok(ch.n < p.N && ch.token + ch.len <= (int64_t)p.B * p.T && blockIdx.x < p.chunks,
                 p.err))
    return;
  auto load = [&](int head, int v) {
    unsigned char *to = shared + S::STAGES + (v & 1) * S::STAGE;
    const Block<KP> w(p, blockIdx.x, head);
    fetch_rows<32, IN>(reinterpret_cast<bf16 *>(to), p.dout, ch, p.H, head, p.V, v * VT);
    fetch_rows<32, IN>(reinterpret_cast<bf16 *>(to + S::V_), p.v, ch, p.H, head, p.V, v * VT);
    to += 2 * S::V_;
    fetch<IN>(to, w.dr(v), S::ROWS);
    fetch<IN>(to + S::ROWS, w.n(v), S::ROWS);
    fetch<IN>(to + 2 * S::ROWS, w.h(v), S::STATE);
    fetch<IN>(to + 2 * S::ROWS + S::STATE, w.D(v), S::STATE);
    ptx::cp_async_commit();
  };
  fetch_rows<KP, IN>(q, p.q, ch, p.Hg, hk, p.K, 0);
  fetch_rows<KP, IN>(k, p.k, ch, p.Hg, hk, p.K, 0);
  load(hk * rep, 0);
  for (int head = hk * rep; head < (hk + 1) * rep; ++head) {
    const Block<KP> w(p, blockIdx.x, head);
    if (tid < 2 * Q) sc[tid] = w.sc()[tid];
    float xq[NT][4] = {}, xk[NT][4] = {}, xs[NT][4] = {}, dP[2][4] = {}, dA[2][4] = {};
    float dot_v = 0.f, dot_h = 0.f;
    for (int v = 0; v < tiles; ++v) {
      const unsigned char *in = shared + S::STAGES + (v & 1) * S::STAGE;
      const bf16 *go = reinterpret_cast<const bf16 *>(in);
      const bf16 *val = reinterpret_cast<const bf16 *>(in + S::V_);
      const bf16 *dr = reinterpret_cast<const bf16 *>(in + 2 * S::V_), *nn = dr + 2 * Q * VT;
      const bf16 *h = nn + 2 * Q * VT, *D = h + 2 * KP * VT;
      ptx::cp_async_wait<0>();
      __syncthreads();  // this tile is here, the one before has been read
      if (v + 1 < tiles) load(head, v + 1);
#pragma unroll
      for (int kk = 0; kk < VT; kk += 16) {
        uint32_t o[4], r[4], rl[4], b[4], bl[4];
        lda<32>(o, go, 16 * wm, kk);
        lda<32>(r, dr, 16 * wm, kk);
        lda<32>(rl, dr + Q * VT, 16 * wm, kk);
        ldb<32>(b, nn, 16 * wn, kk);
        ldb<32>(bl, nn + Q * VT, 16 * wn, kk);
        mma2(dP, o, b);
        mma2(dA, r, b);
        mma2(dP, o, bl);
        mma2(dA, r, bl);
        mma2(dA, rl, b);
#pragma unroll
        for (int j = 0; j < NT; j += 2) {
          ldb<32>(b, h, 8 * (NT * wn + j), kk);
          ldb<32>(bl, h + KP * VT, 8 * (NT * wn + j), kk);
          mma2(xq + j, o, b);
          mma2(xk + j, r, b);
          mma2(xq + j, o, bl);
          mma2(xk + j, r, bl);
          mma2(xk + j, rl, b);
        }
        lda<32>(r, nn, 16 * wm, kk);
        lda<32>(rl, nn + Q * VT, 16 * wm, kk);
#pragma unroll
        for (int j = 0; j < NT; j += 2) {
          ldb<32>(b, D, 8 * (NT * wn + j), kk);
          ldb<32>(bl, D + KP * VT, 8 * (NT * wn + j), kk);
          mma2(xs + j, r, b);
          mma2(xs + j, r, bl);
          mma2(xs + j, rl, b);
        }
      }
      {  // dv = beta dr, dr.v and <h, D>
        const int row = tid >> 3, col = (tid & 7) * 4, place = at<32>(row, col);
        const float b = sc[Q + row];
        float d[4];
#pragma unroll
        for (int e = 0; e < 4; e += 2) {
          const float2 hi = get_pair(dr, place + e), lo = get_pair(dr + Q * VT, place + e);
          const float2 u = get_pair(val, place + e);
          d[e] = hi.x + lo.x;
          d[e + 1] = hi.y + lo.y;
          dot_v = fmaf(d[e], u.x, fmaf(d[e + 1], u.y, dot_v));
        }
        if (row < ch.len && v * VT + col < p.V) {
          __nv_bfloat162 out[2] = {__floats2bfloat162_rn(b * d[0], b * d[1]),
                                   __floats2bfloat162_rn(b * d[2], b * d[3])};
          *reinterpret_cast<uint2 *>(static_cast<bf16 *>(p.dv) +
                                     ((ch.token + row) * p.H + head) * p.V + v * VT + col) =
              *reinterpret_cast<const uint2 *>(out);
        }
        if (tid * 8 < KP * VT)
#pragma unroll
          for (int e = 0; e < 8; e += 2) {
            const float2 a = get_pair(h, tid * 8 + e), al = get_pair(h + KP * VT, tid * 8 + e);
            const float2 c = get_pair(D, tid * 8 + e), cl = get_pair(D + KP * VT, tid * 8 + e);
            dot_h = fmaf(a.x + al.x, c.x + cl.x, fmaf(a.y + al.y, c.y + cl.y, dot_h));
          }
      }
    }
    __syncthreads();  // every tile has been read: dP L and dA L beta take the second's place
    if (head + 1 < (hk + 1) * rep) load(head + 1, 0);
    const float *G = sc, *beta = sc + Q;
    const float GL = G[Q - 1];
    bf16 *PL = reinterpret_cast<bf16 *>(shared + S::STAGES + S::STAGE), *AL = PL + 2 * Q * Q;
    // the terms with h and D, and their products with q and k
    {
      float a[2] = {}, b[2] = {}, c[2] = {};
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        const int row = 16 * wm + g + 8 * e;
        const float fq = p.scale * __expf(G[row]), fk = -__expf(G[row]), fs = __expf(GL - G[row]);
#pragma unroll
        for (int j = 0; j < NT; ++j) {
          const int place = at<KP>(row, 8 * (NT * wn + j) + 2 * t);
          const float2 x = get_pair(q, place), y = get_pair(k, place);
#pragma unroll
          for (int u = 0; u < 2; ++u) {
            float &dq = xq[j][2 * e + u], &dk = xk[j][2 * e + u];
            const float ks = fs * xs[j][2 * e + u], yu = u ? y.y : y.x;
            dq *= fq;
            dk *= fk;
            a[e] = fmaf(dq, u ? x.y : x.x, a[e]);
            b[e] = fmaf(dk, yu, b[e]);
            c[e] = fmaf(ks, yu, c[e]);
            dk = fmaf(beta[row], dk, ks);
          }
        }
      }
      put_rows(qd + wn * Q, 16 * wm + g, t, a[0], a[1]);
      put_rows(kh + wn * Q, 16 * wm + g, t, b[0], b[1]);
      put_rows(kD + wn * Q, 16 * wm + g, t, c[0], c[1]);
    }
    // q k^T and k k^T where this warp has dP and dA
    {
      float sq[2][4] = {}, sk[2][4] = {};
      if (wn <= wm)
#pragma unroll
        for (int kk = 0; kk < KP; kk += 16) {
          uint32_t a[4], b[4];
          ldb<KP>(b, k, 16 * wn, kk);
          lda<KP>(a, q, 16 * wm, kk);
          mma2(sq, a, b);
          lda<KP>(a, k, 16 * wm, kk);
          mma2(sk, a, b);
        }
      float m[2] = {}, bb[2] = {}, cols[2][2] = {};
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        const int row = 16 * wm + g + 8 * e;
#pragma unroll
        for (int j = 0; j < 2; ++j) {
          const int col = 16 * wn + 8 * j + 2 * t;
          float pl[2], al[2];
#pragma unroll
          for (int u = 0; u < 2; ++u) {
            const bool in = row >= col + u && row < ch.len;
            const float L = in ? __expf(G[row] - G[col + u]) : 0.f;
            const float Ls = row == col + u ? 0.f : L;
            pl[u] = in ? L * p.scale * dP[j][2 * e + u] : 0.f;
            const float x = in ? -Ls * dA[j][2 * e + u] : 0.f, B = x * sk[j][2 * e + u];
            al[u] = beta[row] * x;
            const float M = fmaf(pl[u], sq[j][2 * e + u], beta[row] * B);
            m[e] += M;
            bb[e] += B;
            cols[j][u] += M;
          }
          put_pair(PL, PL + Q * Q, at<64>(row, col), pl[0], pl[1]);
          put_pair(AL, AL + Q * Q, at<64>(row, col), al[0], al[1]);
        }
      }
      put_rows(rM + wn * Q, 16 * wm + g, t, m[0], m[1]);
      put_rows(rB + wn * Q, 16 * wm + g, t, bb[0], bb[1]);
#pragma unroll
      for (int j = 0; j < 2; ++j)
#pragma unroll
        for (int u = 0; u < 2; ++u) {
          float x = cols[j][u];
#pragma unroll
          for (int o = 4; o < 32; o <<= 1) x += __shfl_xor_sync(~0u, x, o);
          if (g == 0) cM[wm * Q + 16 * wn + 8 * j + 2 * t + u] = x;
        }
    }
    dot_v += __shfl_xor_sync(~0u, dot_v, 1);
    dot_v += __shfl_xor_sync(~0u, dot_v, 2);
    dot_v += __shfl_xor_sync(~0u, dot_v, 4);
    if ((tid & 7) == 0) rv[tid >> 3] = dot_v;
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) dot_h += __shfl_xor_sync(~0u, dot_h, o);
    if (lane == 0) hD[warp] = dot_h;
    __syncthreads();
    // dq += PL k, dk += AL k + AL^T k + PL^T q; what is zero above or below is skipped
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      uint32_t a[4], al[4], b[4];
      auto add = [&](float (*c)[4], const bf16 *rows) {
#pragma unroll
        for (int j = 0; j < NT; j += 2) {
          ldb_t<KP>(b, rows, 8 * (NT * wn + j), 16 * i);
          mma2(c + j, a, b);
          mma2(c + j, al, b);
        }
      };
      if (i <= wm) {
        lda<64>(a, PL, 16 * wm, 16 * i);
        lda<64>(al, PL + Q * Q, 16 * wm, 16 * i);
        add(xq, k);
        lda<64>(a, AL, 16 * wm, 16 * i);
        lda<64>(al, AL + Q * Q, 16 * wm, 16 * i);
        add(xk, k);
      }
      if (i >= wm) {
        lda_t<64>(a, AL, 16 * wm, 16 * i);
        lda_t<64>(al, AL + Q * Q, 16 * wm, 16 * i);
        add(xk, k);
        lda_t<64>(a, PL, 16 * wm, 16 * i);
        lda_t<64>(al, PL + Q * Q, 16 * wm, 16 * i);
        add(xk, q);
      }
    }
    if (GROUPED) {  // thread by thread: totals [2][NT * 4][IN]
      float *total = reinterpret_cast<float *>(shared + S::TOTALS) + tid;
#pragma unroll
      for (int j = 0; j < NT; ++j)
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          float *a = total + (4 * j + e) * IN, *b = a + 4 * NT * IN;
          if (head > hk * rep) {
            xq[j][e] += *a;
            xk[j][e] += *b;
          }
          *a = xq[j][e];
          *b = xk[j][e];
        }
    }
    if (!GROUPED || head + 1 == (hk + 1) * rep)
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        const int row = 16 * wm + g + 8 * e;
        if (row >= ch.len) continue;
        const int64_t place = ((ch.token + row) * p.Hg + hk) * p.K;
#pragma unroll
        for (int j = 0; j < NT; ++j) {
          const int col = 8 * (NT * wn + j) + 2 * t;
          if (col >= p.K) continue;
          *reinterpret_cast<__nv_bfloat162 *>(static_cast<bf16 *>(p.dq) + place + col) =
              __floats2bfloat162_rn(xq[j][2 * e], xq[j][2 * e + 1]);
          *reinterpret_cast<__nv_bfloat162 *>(static_cast<bf16 *>(p.dk) + place + col) =
              __floats2bfloat162_rn(xk[j][2 * e], xk[j][2 * e + 1]);
        }
      }
    if (warp == 0) {  // dbeta, and dG summed from the end: lane l has tokens l and l + 32
      float d[2], all = 0.f, state = lane < IN / 32 ? hD[lane] : 0.f;
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        const int i = lane + 32 * e;
        auto quarters = [&](const float *x) { return x[i] + x[Q + i] + x[2 * Q + i] + x[3 * Q + i]; };
        const float kd = quarters(kD), khi = quarters(kh);
        d[e] = quarters(rM) - quarters(cM) + quarters(qd) + beta[i] * khi - kd;
        all += kd;
        if (i < ch.len) p.dbeta[(ch.token + i) * p.H + head] = rv[i] + khi + quarters(rB);
      }
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) {
        all += __shfl_xor_sync(~0u, all, o);
        state += __shfl_xor_sync(~0u, state, o);
      }
      const float end = fmaf(__expf(GL), state, all);
#pragma unroll
      for (int e = 0; e < 2; ++e)
        if (lane + 32 * e == ch.len - 1) d[e] += end;
      if (!p.g_is_cumsum) {
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
          const float a = __shfl_down_sync(~0u, d[0], o), b = __shfl_down_sync(~0u, d[1], o);
          if (lane + o < 32) {
            d[0] += a;
            d[1] += b;
          }
        }
        d[0] += __shfl_sync(~0u, d[1], 0);
      }
#pragma unroll
      for (int e = 0; e < 2; ++e)
        if (lane + 32 * e < ch.len) p.dg[(ch.token + lane + 32 * e) * p.H + head] = d[e];
    }
    __syncthreads();  // the sums and the second stage are free
  }
}

template <int KP>
cudaError_t launch(const DeltaBwdParams &p, cudaStream_t stream) {
  auto room = [](const void *kernel, int bytes) {
    return cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
  };
  const bool grouped = p.H > p.Hg;
  const void *inputs = grouped ? reinterpret_cast<const void *>(tc_inputs_kernel<KP, true>)
                               : reinterpret_cast<const void *>(tc_inputs_kernel<KP, false>);
  cudaError_t e = room(reinterpret_cast<const void *>(tc_prepare_kernel<KP>), PrepareShared<KP>::BYTES);
  if (e == cudaSuccess)
    e = room(reinterpret_cast<const void *>(tc_states_kernel<KP>), StatesShared<KP>::BYTES);
  if (e == cudaSuccess)
    e = room(reinterpret_cast<const void *>(tc_grads_kernel<KP>), GradsShared<KP>::BYTES);
  if (e == cudaSuccess) e = room(inputs, InputsShared<KP>::bytes(grouped));
  if (e != cudaSuccess) return e;
  const dim3 chunks((unsigned)p.chunks, p.H), walks((p.V + VT - 1) / VT, p.H, p.N);
  tc_prepare_kernel<KP><<<chunks, PREP, PrepareShared<KP>::BYTES, stream>>>(p);
  tc_states_kernel<KP><<<walks, WALK, StatesShared<KP>::BYTES, stream>>>(p);
  tc_grads_kernel<KP><<<walks, WALK, GradsShared<KP>::BYTES, stream>>>(p);
  const dim3 keys((unsigned)p.chunks, p.Hg);
  if (grouped)
    tc_inputs_kernel<KP, true><<<keys, IN, InputsShared<KP>::bytes(true), stream>>>(p);
  else
    tc_inputs_kernel<KP, false><<<keys, IN, InputsShared<KP>::bytes(false), stream>>>(p);
  return cudaGetLastError();
}

}  // namespace

bool delta_bwd_tc_supported(const DeltaBwdParams &p, bool bf16) {
  return bf16 && p.K % 8 == 0 && p.V % 8 == 0 && p.K <= 128 && p.V <= 128;
}

int64_t delta_bwd_tc_block(const DeltaBwdParams &p) {
  const int tiles = (p.V + VT - 1) / VT;
  return p.K <= 64 ? Block<64>::bytes(tiles) : Block<128>::bytes(tiles);
}

cudaError_t launch_delta_bwd_tc(const DeltaBwdParams &p, cudaStream_t stream) {
  return p.K <= 64 ? launch<64>(p, stream) : launch<128>(p, stream);
}

}  // namespace gdn
