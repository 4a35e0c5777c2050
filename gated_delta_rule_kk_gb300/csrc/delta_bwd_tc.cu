// The gated delta rule's gradient over chunks on the tensor cores: bfloat16 inputs, K and V
// multiples of 8, K <= 128, V <= 128.  Here what every chunk does by itself: T and P at the
// beginning, the inputs' gradients at the end; the walks over the chunks between them are in
// delta_bwd_walk.cu.
#include <algorithm>

#include "delta_bwd_tc.cuh"

namespace gdn {
namespace {

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
    w.sc()[2 * Q + tid] = expf(G[tid]);
    w.sc()[3 * Q + tid] = expf(G[Q - 1] - G[tid]);
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

// ---------------------------------------------------------------- the inputs' gradients

constexpr int IN = 512;

template <int KP>
struct InputsShared {
  static constexpr int K_ = Q * KP * 2, V_ = Q * VT * 2;
  static constexpr int ROWS = Block<KP>::ROWS, STATE = Block<KP>::STATE;
  // a value tile: do, v, dr, n, h, D; the second one's place then holds dP L and dA L beta
  static constexpr int STAGE = std::max(2 * V_ + 2 * ROWS + 2 * STATE, 2 * Block<KP>::SQUARE);
  static constexpr int STAGES = 2 * K_, SUMS = STAGES + 2 * STAGE;
  static constexpr int SUM_FLOATS = (24 + IN / 32 + 4) * Q + IN / 32;
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
  // by quarters: q.dq_h, k.dk_h / beta, k.dk_s, rows of M, rows of B; columns of M by wm;
  // dr.v by warps
  float *qd = sums, *kh = qd + 4 * Q, *kD = kh + 4 * Q, *rM = kD + 4 * Q, *rB = rM + 4 * Q;
  float *cM = rB + 4 * Q, *rv = cM + 4 * Q, *sc = rv + IN / 32 * Q, *hD = sc + 4 * Q;
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
    if (tid < 4 * Q) sc[tid] = w.sc()[tid];
    float xq[NT][4] = {}, xk[NT][4] = {}, xs[NT][4] = {}, dP[2][4] = {}, dA[2][4] = {};
    float dot_v[2] = {}, dot_h = 0.f;
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
        lda_tiles<Q>(r, dr, 16 * wm, kk);
        lda_tiles<Q>(rl, dr + Q * VT, 16 * wm, kk);
        ldb_tiles<Q>(b, nn, 16 * wn, kk);
        ldb_tiles<Q>(bl, nn + Q * VT, 16 * wn, kk);
        mma2(dP, o, b);
        mma2(dA, r, b);
        mma2(dP, o, bl);
        mma2(dA, r, bl);
        mma2(dA, rl, b);
#pragma unroll
        for (int j = 0; j < NT; j += 2) {
          ldb_tiles<KP>(b, h, 8 * (NT * wn + j), kk);
          ldb_tiles<KP>(bl, h + KP * VT, 8 * (NT * wn + j), kk);
          mma2(xq + j, o, b);
          mma2(xk + j, r, b);
          mma2(xq + j, o, bl);
          mma2(xk + j, r, bl);
          mma2(xk + j, rl, b);
        }
        lda_tiles<Q>(r, nn, 16 * wm, kk);
        lda_tiles<Q>(rl, nn + Q * VT, 16 * wm, kk);
#pragma unroll
        for (int j = 0; j < NT; j += 2) {
          ldb_tiles<KP>(b, D, 8 * (NT * wn + j), kk);
          ldb_tiles<KP>(bl, D + KP * VT, 8 * (NT * wn + j), kk);
          mma2(xs + j, r, b);
          mma2(xs + j, r, bl);
          mma2(xs + j, rl, b);
        }
      }
      {  // dr.v and <h, D>; a warp has two value columns, a lane two tokens
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          const int c = 2 * warp + e, place = (c / 8 * (Q / 8) + lane / 4) * 64 + c % 8 * 8 + lane % 4 * 2;
          const float2 hi = get_pair(dr, place), lo = get_pair(dr + Q * VT, place);
          dot_v[0] = fmaf(hi.x + lo.x, to_f32(val[at<32>(2 * lane, c)]), dot_v[0]);
          dot_v[1] = fmaf(hi.y + lo.y, to_f32(val[at<32>(2 * lane + 1, c)]), dot_v[1]);
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
    const float *G = sc, *beta = sc + Q, *eG = sc + 2 * Q, *eR = sc + 3 * Q;
    bf16 *PL = reinterpret_cast<bf16 *>(shared + S::STAGES + S::STAGE), *AL = PL + 2 * Q * Q;
    // the terms with h and D, and their products with q and k
    {
      float a[2] = {}, b[2] = {}, c[2] = {};
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        const int row = 16 * wm + g + 8 * e;
        const float fq = p.scale * eG[row], fk = -eG[row], fs = eR[row];
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
    *reinterpret_cast<float2 *>(rv + warp * Q + 2 * lane) = make_float2(dot_v[0], dot_v[1]);
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
        float v = 0.f;
#pragma unroll
        for (int u = 0; u < IN / 32; ++u) v += rv[u * Q + i];
        if (i < ch.len) p.dbeta[(ch.token + i) * p.H + head] = v + khi + quarters(rB);
      }
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) {
        all += __shfl_xor_sync(~0u, all, o);
        state += __shfl_xor_sync(~0u, state, o);
      }
      const float end = fmaf(eG[Q - 1], state, all);
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
  if (e == cudaSuccess) e = room(inputs, InputsShared<KP>::bytes(grouped));
  if (e != cudaSuccess) return e;
  const dim3 chunks((unsigned)p.chunks, p.H);
  tc_prepare_kernel<KP><<<chunks, PREP, PrepareShared<KP>::BYTES, stream>>>(p);
  e = cudaGetLastError();
  if (e == cudaSuccess) e = launch_delta_walks(p, stream);
  if (e != cudaSuccess) return e;
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
