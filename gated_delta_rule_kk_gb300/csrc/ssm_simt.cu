// The state space scan over prompts in float32 on the CUDA cores, for every
// type and size: the recurrence token by token,
//   h = e^(a s_t) h + (s_t x_t) B_t^T,   y_t = h C_t + D x_t,   a = -e^A_log,
// with the state in registers.
//
// A block of 128 threads owns 32 rows of one head's state for one segment:
// eight lanes share a row (each 4 of every 32 columns), a thread holds two
// rows.  Tokens come in blocks of 32 through shared memory, widened to
// float32.  Per token a thread takes three operations for each of its state
// elements (two lanes an instruction) and sums two outputs over eight lanes;
// that arithmetic, one token after another, is what bounds it (4096 tokens, 64
// heads of 64 x 128, float32: 619 us in segments, 13.9 TFLOP/s of the recurrence's
// four operations; 773 tokens, 12 heads of 40 x 48: 31 us).
//
// When sequences are cut into segments the kernel runs twice: first every
// segment but a sequence's last from zero, keeping its last state and decay,
// then every segment from its start, which it forms from the sequence's
// segments before it.
#include <type_traits>

#include "rows.cuh"
#include "ssm_items.cuh"

namespace gdn {
namespace {

constexpr int SS_TB = 32;    // tokens of a block
constexpr int SS_ROWS = 32;  // state rows of a block
constexpr int SS_THREADS = 128;

template <int KJ>
struct SsmSmem {
  static constexpr int KP = 32 * KJ;
  float B[SS_TB][KP], C[SS_TB][KP];
  float x[SS_TB][SS_ROWS], y[SS_TB][SS_ROWS];
  float in[SS_TB], out[SS_TB], decay[SS_TB];  // factors of x and of y, decay
  float total;                                // the block's log-decay
  int scaled;
};

constexpr float SS_MOST = 16.f;  // |G| of a block that is held scaled

// KJ: float4 columns of a lane, K <= 32 KJ.  STATES: the first of two passes.
template <typename T, int KJ, bool STATES>
__global__ void __launch_bounds__(SS_THREADS) ssm_simt_kernel(SsmParams p) {
  extern __shared__ __align__(16) unsigned char smem_raw[];
  SsmSmem<KJ> &sm = *reinterpret_cast<SsmSmem<KJ> *>(smem_raw);
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int kl = tid & 7, r0 = tid >> 3;
  const int item = blockIdx.x, h = blockIdx.y, v0 = blockIdx.z * SS_ROWS;
  if (!offsets_ok(p.cu, p.N, p.T, p.err)) return;
  const SsmItem q = ssm_item(p, item);
  if (q.n < 0 || (STATES && q.last)) return;
  if (!bounds_ok(q.n < p.N && q.lo >= 0 && q.lo <= q.hi && q.hi <= p.T && h < p.H && v0 < p.V, p.err))
    return;
  const int K = p.K, V = p.V, g = h / (p.H / p.Hg);
  const float a = -expf(p.A_log[h]), bias = p.dt_bias ? p.dt_bias[h] : 0.f;
  const int64_t xat = q.b * p.xb + (int64_t)h * V, bat = q.b * p.bb + (int64_t)g * K;
  const int64_t cat = q.b * p.cb + (int64_t)g * K, zat = q.b * p.zb + (int64_t)h * V;
  const int64_t yat = q.b * p.yb + (int64_t)h * V, dat = q.b * p.dtb;

  // rows v0 + r0 and v0 + r0 + 16, columns 32 j + 4 kl ..
  float s[2][4 * KJ];
  auto column = [&](int j, int e) { return 32 * j + 4 * kl + e; };
  auto load_state = [&](const float *src, float (&out)[2][4 * KJ]) {
#pragma unroll
    for (int r = 0; r < 2; ++r) {
      const int v = v0 + r0 + 16 * r;
#pragma unroll
      for (int i = 0; i < 4 * KJ; ++i) {
        const int k = column(i / 4, i % 4);
        out[r][i] = src && v < V && k < K ? src[(int64_t)v * K + k] : 0.f;
      }
    }
  };
  const int64_t tile = (int64_t)V * K;
  load_state(!STATES && p.h0 ? p.h0 + ((int64_t)q.n * p.H + h) * tile : nullptr, s);
  if (!STATES) {
    for (int i = q.first; i < item; ++i) {
      float add[2][4 * KJ];
      load_state(p.seg_state + ((int64_t)i * p.H + h) * tile, add);
      const float d = expf(p.seg_decay[(int64_t)i * p.H + h]);
#pragma unroll
      for (int r = 0; r < 2; ++r)
#pragma unroll
        for (int e = 0; e < 4 * KJ; ++e) s[r][e] = fmaf(d, s[r][e], add[r][e]);
    }
  }
  // columns past K stay zero
  for (int i = tid; i < SS_TB * SsmSmem<KJ>::KP; i += SS_THREADS) {
    (&sm.B[0][0])[i] = 0.f;
    (&sm.C[0][0])[i] = 0.f;
  }
  for (int i = tid; i < SS_TB * SS_ROWS; i += SS_THREADS) (&sm.x[0][0])[i] = 0.f;
  float total = 0.f;
  for (int t0 = q.lo; t0 < q.hi; t0 += SS_TB) {
    const int n = min(SS_TB, q.hi - t0);
    __syncthreads();
    // rows past the last token, up to a whole four, are left as they are: finite,
    // and taken with factors of zero
    for (int i = warp; i < n; i += 4) {
      const T *bt = static_cast<const T *>(p.Bm) + bat + (int64_t)(t0 + i) * p.bs;
      const T *ct = static_cast<const T *>(p.Cm) + cat + (int64_t)(t0 + i) * p.cs;
      const T *xt = static_cast<const T *>(p.x) + xat + (int64_t)(t0 + i) * p.xs;
#pragma unroll
      for (int j = 0; j < KJ; ++j) {
        const int k = 32 * j + lane;
        if (k >= K) continue;
        sm.B[i][k] = to_f32(bt[k]);
        if (!STATES) sm.C[i][k] = to_f32(ct[k]);
      }
      sm.x[i][lane] = v0 + lane < V ? to_f32(xt[v0 + lane]) : 0.f;
    }
    if (warp == 0) {
      const float step = lane < n ? ssm_step(p, dat + (int64_t)(t0 + lane) * p.dts, h, bias) : 0.f;
      const float own = a * step;
      float G = own;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const float v = __shfl_up_sync(~0u, G, o);
        if (lane >= o) G += v;
      }
      const bool scaled = __all_sync(~0u, fabsf(G) <= SS_MOST);
      sm.in[lane] = scaled ? step * expf(-G) : step;
      sm.out[lane] = scaled ? expf(G) : 1.f;
      sm.decay[lane] = expf(own);
      if (lane == 31) {
        sm.total = G;
        sm.scaled = scaled;
      }
    }
    __syncthreads();
    total += sm.total;
    // Four tokens at a time: their eight partial outputs (of two rows) are summed
    // over the row's eight lanes together, halving values and lanes at each step,
    // and lane kl ends with token kl / 2's row kl % 2.  Tokens past the block's
    // last have factors of zero and a decay of one.
    auto tokens = [&](auto scaled) {
#pragma unroll 1
      for (int i = 0; i < n; i += 4) {
        float sum[8];
#pragma unroll
        for (int t = 0; t < 4; ++t) {
          float acc[2][4] = {}, in[2];
          const float d = sm.decay[i + t];
          const float dd[4] = {d, d, d, d};
#pragma unroll
          for (int r = 0; r < 2; ++r) in[r] = sm.in[i + t] * sm.x[i + t][r0 + 16 * r];
#pragma unroll
          for (int j = 0; j < KJ; ++j) {
            const float4 b4 = *reinterpret_cast<const float4 *>(&sm.B[i + t][32 * j + 4 * kl]);
            const float bv[4] = {b4.x, b4.y, b4.z, b4.w};
            float cv[4];
            if (!STATES) {
              const float4 c4 = *reinterpret_cast<const float4 *>(&sm.C[i + t][32 * j + 4 * kl]);
              cv[0] = c4.x; cv[1] = c4.y; cv[2] = c4.z; cv[3] = c4.w;
            }
#pragma unroll
            for (int r = 0; r < 2; ++r) {
              float *h4 = &s[r][4 * j];
              if constexpr (decltype(scaled)::value) {
                const float ii[4] = {in[r], in[r], in[r], in[r]};
                fma_row<4>(h4, ii, bv);
              } else {
                float add[4] = {in[r] * bv[0], in[r] * bv[1], in[r] * bv[2], in[r] * bv[3]};
                fma_row<4>(add, dd, h4);
#pragma unroll
                for (int e = 0; e < 4; ++e) h4[e] = add[e];
              }
              if (!STATES) fma_row<4>(acc[r], h4, cv);
            }
          }
#pragma unroll
          for (int r = 0; r < 2; ++r)
            sum[2 * t + r] = (acc[r][0] + acc[r][1]) + (acc[r][2] + acc[r][3]);
        }
        if (!STATES) {
#pragma unroll
          for (int m = 4, o = 4; o > 0; m /= 2, o /= 2) {
            const bool up = kl & o;
#pragma unroll
            for (int j = 0; j < m; ++j) {
              const float send = up ? sum[j] : sum[j + m], keep = up ? sum[j + m] : sum[j];
              sum[j] = keep + __shfl_xor_sync(~0u, send, o);
            }
          }
          const int t = i + kl / 2;
          sm.y[t][r0 + 16 * (kl & 1)] = sm.out[t] * sum[0];
        }
      }
    };
    if (sm.scaled) {
      tokens(std::true_type());
      const float d = expf(sm.total);
#pragma unroll
      for (int r = 0; r < 2; ++r)
#pragma unroll
        for (int e = 0; e < 4 * KJ; ++e) s[r][e] *= d;
    } else {
      tokens(std::false_type());
    }
    if (!STATES) {
      __syncthreads();
      const int v = v0 + lane;
      if (v < V) {
        const float skip = p.D ? p.D[h] : 0.f;
        for (int i = warp; i < n; i += 4) {
          float y = fmaf(skip, sm.x[i][lane], sm.y[i][lane]);
          if (p.z)
            y *= silu(to_f32(static_cast<const T *>(p.z)[zat + (int64_t)(t0 + i) * p.zs + v]));
          const int64_t at = yat + (int64_t)(t0 + i) * p.ys + v;
          if (p.y_f32)
            static_cast<float *>(p.y)[at] = y;
          else
            static_cast<T *>(p.y)[at] = from_f32<T>(y);
        }
      }
    }
  }
  float *dst = nullptr;
  if (STATES) {
    dst = p.seg_state + ((int64_t)item * p.H + h) * tile;
    if (tid == 0 && v0 == 0) p.seg_decay[(int64_t)item * p.H + h] = total;
  } else if (q.last && p.ht) {
    dst = p.ht + ((int64_t)q.n * p.H + h) * tile;
  }
  if (dst == nullptr) return;
#pragma unroll
  for (int r = 0; r < 2; ++r) {
    const int v = v0 + r0 + 16 * r;
#pragma unroll
    for (int i = 0; i < 4 * KJ; ++i) {
      const int k = column(i / 4, i % 4);
      if (v < V && k < K) dst[(int64_t)v * K + k] = s[r][i];
    }
  }
}

template <typename T, int KJ>
cudaError_t launch(const SsmParams &p, cudaStream_t stream) {
  const dim3 grid((unsigned)p.items, (unsigned)p.H, (unsigned)((p.V + SS_ROWS - 1) / SS_ROWS));
  constexpr size_t bytes = sizeof(SsmSmem<KJ>);
  if (p.seg_state) {
    const cudaError_t e = cudaFuncSetAttribute(
        ssm_simt_kernel<T, KJ, true>, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)bytes);
    if (e != cudaSuccess) return e;
    ssm_simt_kernel<T, KJ, true><<<grid, SS_THREADS, bytes, stream>>>(p);
  }
  const cudaError_t e = cudaFuncSetAttribute(
      ssm_simt_kernel<T, KJ, false>, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)bytes);
  if (e != cudaSuccess) return e;
  ssm_simt_kernel<T, KJ, false><<<grid, SS_THREADS, bytes, stream>>>(p);
  return cudaGetLastError();
}

template <typename T>
cudaError_t launch_k(const SsmParams &p, cudaStream_t stream) {
  if (p.K <= 32) return launch<T, 1>(p, stream);
  if (p.K <= 64) return launch<T, 2>(p, stream);
  if (p.K <= 128) return launch<T, 4>(p, stream);
  return launch<T, 8>(p, stream);
}

}  // namespace

cudaError_t launch_ssm_simt(const SsmParams &p, bool bf16, cudaStream_t stream) {
  return bf16 ? launch_k<__nv_bfloat16>(p, stream) : launch_k<float>(p, stream);
}

}  // namespace gdn
