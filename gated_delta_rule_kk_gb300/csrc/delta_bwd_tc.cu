// The gated delta rule's gradient over chunks on the tensor cores: bfloat16 inputs, K and V
// multiples of 8, K <= 128, V <= 128.  Here T and P of every chunk; the walks over the chunks
// are in delta_bwd_walk.cu, the inputs' gradients in delta_bwd_inputs.cu.
#include "delta_bwd_tc.cuh"

namespace gdn {
namespace {

// grid: chunks, heads.  Running log-gates, P, A and T = (I + A)^-1.  [q; k] k^T on the tensor
// cores.  The inverse: the four 16 x 16 blocks on the diagonal by forward substitution in
// float32, a column a thread; then the blocks below it, a diagonal at a time and a warp a
// block, T_(b+d, b) = -T_(b+d, b+d) sum_m A_(b+d, m) T_(m, b), as products of pairs of
// bfloat16 pieces: transposed, so that the sum's accumulators are the left operand of the
// product behind it.  (As float32 sums from shared memory, two loads a multiplication, they
// took a third of the kernel's instructions: 80 us at 2 x 4096 tokens, 16 heads of 128; then 53.
// Now 55: the sums' rests.)
// Barriers between the phases are what a warp waits for most: four blocks an SM, T in the place
// of the images before it (three blocks: 59 us).
constexpr int PREP = 256;
template <int KP>
struct PrepareShared {
  static constexpr int PITCH = Q + 8;  // of A and T in float32
  // q and k, then P's and A's images, then T and behind it its image; A
  static constexpr int T_IMAGE = Q * PITCH * 4, IMAGES = T_IMAGE + Block<KP>::SQUARE;
  static constexpr int BYTES = IMAGES + (Q * PITCH + 3 * Q) * 4;
  static_assert(IMAGES >= 2 * Block<KP>::SQUARE && IMAGES >= 2 * Q * KP * 2, "");
};

template <int KP>
__global__ void __launch_bounds__(PREP, 4) tc_prepare_kernel(DeltaBwdParams p) {
  extern __shared__ __align__(128) unsigned char shared[];
  ptx::griddep_wait();
  bf16 *q = reinterpret_cast<bf16 *>(shared), *k = q + Q * KP;
  constexpr int PITCH = PrepareShared<KP>::PITCH;
  float(*A)[PITCH] = reinterpret_cast<float(*)[PITCH]>(shared + PrepareShared<KP>::IMAGES);
  float(*T)[PITCH] = reinterpret_cast<float(*)[PITCH]>(shared);
  float2 *G = reinterpret_cast<float2 *>(A + Q);  // sums and their rests
  float *beta = reinterpret_cast<float *>(G + Q);
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
    float g[2], less[2] = {0.f, 0.f};
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      const int i = lane + 32 * e;
      const int64_t where = (ch.token + min(i, ch.len - 1)) * p.H + head;
      g[e] = i < ch.len || p.g_is_cumsum ? p.g[where] : 0.f;
      if (!p.g_is_cumsum) g[e] = delta_gate(g[e]);
      beta[i] = i < ch.len ? p.beta[where] : 0.f;
    }
    if (!p.g_is_cumsum) {
      double sum[2] = {g[0], g[1]};
#pragma unroll
      for (int e = 0; e < 2; ++e)
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
          const double v = __shfl_up_sync(~0u, sum[e], o);
          if (lane >= o) sum[e] += v;
        }
      sum[1] += __shfl_sync(~0u, sum[0], 31);
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        g[e] = (float)sum[e];
        less[e] = (float)(sum[e] - g[e]);
      }
    }
    G[lane] = make_float2(g[0], less[0]);
    G[lane + 32] = make_float2(g[1], less[1]);
  }
  ptx::cp_async_wait<0>();
  __syncthreads();
  if (tid < Q) {
    w.sc()[tid] = G[tid].x;
    w.sc()[Q + tid] = beta[tid];
    w.sc()[2 * Q + tid] = expf(G[tid].x);
    w.sc()[3 * Q + tid] = expf(delta_gap(G[Q - 1], G[tid]));
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
  bf16 *Ph = reinterpret_cast<bf16 *>(shared), *Pl = Ph + Q * Q, *Ah = Pl + Q * Q, *Al = Ah + Q * Q;
#pragma unroll
  for (int j = 0; j < 8; ++j)
#pragma unroll
    for (int r = 0; r < 2; ++r) {
      const int row = 16 * wm + g + 8 * r, col = 8 * j + 2 * t;
      float v[2];
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        const bool in = of_q ? row >= col + e : row > col + e;
        v[e] = in ? (of_q ? p.scale : 1.f) * s[j][2 * r + e] * __expf(delta_gap(G[row], G[col + e]))
                  : 0.f;
      }
      if (of_q) {
        put_pair(Ph, Pl, at<64>(row, col), v[0], v[1]);
      } else {
        put_pair(Ah, Al, at<64>(row, col), v[0], v[1]);
        *reinterpret_cast<float2 *>(&A[row][col]) = make_float2(beta[row] * v[0], beta[row] * v[1]);
      }
    }
  __syncthreads();
  keep<PREP>(w.P(), shared, 2 * Block<KP>::SQUARE);
  __syncthreads();  // T takes their place
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
#pragma unroll
  for (int d = 1; d < 4; ++d) {
    if (warp + d < 4) {
      const int b = 16 * warp, i0 = 16 * (warp + d);
      // x^T [j][i] = sum_m T_(m, b)^T A_(b+d, m)^T
      float x[2][4] = {};
#pragma unroll
      for (int m = 0; m < d; ++m) {
        uint32_t ah[4], al[4], bh[4], bl[4];
        const int r0 = b + 16 * m;
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const int r = r0 + 2 * t + 8 * (e >> 1), j = b + g + 8 * (e & 1);
          split(T[r][j], T[r + 1][j], ah[e], al[e]);
          const float2 y = *reinterpret_cast<const float2 *>(&A[i0 + g + 8 * (e >> 1)][r0 + 2 * t + 8 * (e & 1)]);
          split(y.x, y.y, bh[e], bl[e]);
        }
        mma2(x, ah, bh);
        mma2(x, ah, bl);
        mma2(x, al, bh);
      }
      // T_(b+d, b)^T [j][i] = -x^T T_(b+d, b+d)^T
      float y[2][4] = {};
      uint32_t ah[4], al[4], bh[4], bl[4];
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        split(x[e >> 1][e % 2 * 2], x[e >> 1][e % 2 * 2 + 1], ah[e], al[e]);
        const float2 z = *reinterpret_cast<const float2 *>(&T[i0 + g + 8 * (e >> 1)][i0 + 2 * t + 8 * (e & 1)]);
        split(z.x, z.y, bh[e], bl[e]);
      }
      mma2(y, ah, bh);
      mma2(y, ah, bl);
      mma2(y, al, bh);
#pragma unroll
      for (int n = 0; n < 2; ++n)
#pragma unroll
        for (int e = 0; e < 4; ++e) T[i0 + 8 * n + 2 * t + (e & 1)][b + g + 8 * (e >> 1)] = -y[n][e];
    }
    __syncthreads();
  }
  bf16 *Th = reinterpret_cast<bf16 *>(shared + PrepareShared<KP>::T_IMAGE), *Tl = Th + Q * Q;
  for (int i = tid; i < Q * Q / 2; i += PREP) {
    const int row = i / 32, col = i % 32 * 2;
    put_pair(Th, Tl, at<64>(row, col), row >= col ? T[row][col] : 0.f,
             row >= col + 1 ? T[row][col + 1] : 0.f);
    if (row < 8 && col >= 48)
      *reinterpret_cast<float *>(Th + at<64>(row, col)) = G[row * 8 + (col - 48) / 2].y;
  }
  __syncthreads();
  keep<PREP>(w.T(), Th, Block<KP>::SQUARE);
}

template <int KP>
cudaError_t launch(const DeltaBwdParams &p, cudaStream_t stream) {
  constexpr int BYTES = PrepareShared<KP>::BYTES;
  const cudaError_t e = cudaFuncSetAttribute(tc_prepare_kernel<KP>,
                                             cudaFuncAttributeMaxDynamicSharedMemorySize, BYTES);
  if (e != cudaSuccess) return e;
  const dim3 grid((unsigned)p.chunks, p.H);
  if (p.cu != nullptr) return launch_behind(tc_prepare_kernel<KP>, grid, PREP, BYTES, stream, p);
  tc_prepare_kernel<KP><<<grid, PREP, BYTES, stream>>>(p);  // the call's first kernel
  return cudaGetLastError();
}

}  // namespace

// (2 x 4096 tokens, 16 heads, K x V, tensor cores / CUDA cores, us: 128 x 128 465 / 5170,
// 120 x 128 471 / 5090; on CUDA cores 127 x 128 5190, 128 x 136 5090, 128 x 256 5960.  Rows of K
// and V that are no multiples of 8 do not begin on the 16 bytes that the copies want; that V ends
// at 128 is a limit of what was tried, as value tiles do not depend on one another.)
bool delta_bwd_tc_supported(const DeltaBwdParams &p, bool bf16) {
  return bf16 && p.K % 8 == 0 && p.V % 8 == 0 && p.K <= 128 && p.V <= 128;
}

int64_t delta_bwd_tc_block(const DeltaBwdParams &p) {
  const int tiles = (p.V + VT - 1) / VT;
  return p.K <= 64 ? Block<64>::bytes(tiles) : Block<128>::bytes(tiles);
}

cudaError_t launch_delta_bwd_tc(const DeltaBwdParams &p, cudaStream_t stream) {
  cudaError_t e = p.K <= 64 ? launch<64>(p, stream) : launch<128>(p, stream);
  if (e == cudaSuccess) e = launch_delta_walks(p, stream);
  if (e == cudaSuccess) e = launch_delta_inputs(p, stream);
  return e;
}

}  // namespace gdn
