// Gradient of the norm over groups of channels.  With n the normal form, r = 1 / root,
// m = n w + b and dm the gradient of m:
//   z after:  dm = dy act(z), dz = dy m act'(z);   no z: dm = dy act'(m);   z first: dm = dy
//   dw = sum_t dm n,  db = sum_t dm
//   dn = dm w,  du = r (dn - n mean(dn n) - mean(dn))   (the last with the mean taken off)
//   dx = du, or with z first dx = du act(z), dz = du x act'(z)
// One pass: dy, x and z are read once, dx and dz written once.  dw and db are summed over a
// team's tokens in registers, over a block's teams in shared memory and over the blocks by a
// second kernel, each in a fixed order.
#include "group_norm.cuh"

namespace gdn {
namespace {

// Threads of a block: 256, or what the widest groups want (WIDE).
constexpr int bwd_threads(int elements, bool wide) {
  return wide ? norm_threads(elements) : NORM_BWD_THREADS;
}

template <typename T, int VEC, int PP, bool Z, bool WIDE>
__global__ void __launch_bounds__(bwd_threads(PP * VEC, WIDE), WIDE ? 1 : norm_bwd_per_sm(PP * VEC))
norm_bwd_kernel(NormParams p) {
  __shared__ float buf[2][NORM_WARPS][2];
  extern __shared__ float sums[];  // [threads][PP * VEC]
  const NormTeam m(p);
  if (!bounds_ok(p.team * p.rows * p.span <= (int)blockDim.x, p.err)) return;
  int turn = 0;
  const float inv = 1.f / (float)p.W;
  float w[PP][VEC], b[PP][VEC], dw[PP][VEC], db[PP][VEC];
  NormRow<T, VEC, PP> x, z, g;
  x.zero();
  z.zero();
  g.zero();
  g.load(p, m, p.dy, p.gs, p.gb, m.t);
  x.load(p, m, p.x, p.xs, p.xb, m.t);
  if (Z) z.load(p, m, p.z, p.zs, p.zb, m.t);
  norm_weights<T>(p, m, p.weight, 1.f, w);
  norm_weights<T>(p, m, p.bias, 0.f, b);
#pragma unroll
  for (int j = 0; j < PP; ++j)
#pragma unroll
    for (int e = 0; e < VEC; ++e) dw[j][e] = db[j][e] = 0.f;
  const int first = blockIdx.x / p.blocks_per_row * p.rows;
  for (int t0 = first, t = m.t; t0 < p.tokens; t0 += p.step, t += p.step) {
    const bool there = m.live && t < p.tokens;
    float n[PP][VEC], d[PP][VEC], raw[Z ? PP : 1][VEC], zv[Z ? PP : 1][VEC];
#pragma unroll
    for (int j = 0; j < PP; ++j) {
      x.r[j].widen(n[j]);
      g.r[j].widen(d[j]);
      if constexpr (Z) {
        z.r[j].widen(zv[j]);
        if (p.gate_first) {
          float gate[VEC];
          norm_act<VEC>(p.act, zv[j], gate, nullptr);
#pragma unroll
          for (int e = 0; e < VEC; ++e) {
            raw[j][e] = n[j][e];
            n[j][e] *= gate[e];
          }
        }
      }
    }
    g.load(p, m, p.dy, p.gs, p.gb, t + p.step);
    x.load(p, m, p.x, p.xs, p.xb, t + p.step);
    if (Z) z.load(p, m, p.z, p.zs, p.zb, t + p.step);
    const float r = normalise<VEC, PP>(p, m, n, buf, turn);
    float s[2] = {0.f, 0.f};  // of dn n and of dn
    NormRow<T, VEC, PP> out;
#pragma unroll
    for (int j = 0; j < PP; ++j) {
      if constexpr (Z) {
        if (!p.gate_first) {
          float gate[VEC], slope[VEC];
          norm_act<VEC>(p.act, zv[j], gate, slope);
#pragma unroll
          for (int e = 0; e < VEC; ++e) {
            slope[e] *= d[j][e] * fmaf(n[j][e], w[j][e], b[j][e]);
            d[j][e] *= gate[e];
          }
          out.r[j].round(slope);
        }
      } else if (p.act != GDN_ACT_NONE) {
        float v[VEC], slope[VEC];
#pragma unroll
        for (int e = 0; e < VEC; ++e) v[e] = fmaf(n[j][e], w[j][e], b[j][e]);
        norm_act<VEC>(p.act, v, v, slope);
#pragma unroll
        for (int e = 0; e < VEC; ++e) d[j][e] *= slope[e];
      }
#pragma unroll
      for (int e = 0; e < VEC; ++e) {
        if (there) {
          dw[j][e] = fmaf(d[j][e], n[j][e], dw[j][e]);
          db[j][e] += d[j][e];
        }
        d[j][e] *= w[j][e];
        s[0] = fmaf(d[j][e], n[j][e], s[0]);
        s[1] += d[j][e];
      }
    }
    if constexpr (Z)
      if (!p.gate_first) out.store(p, m, p.dz, p.ds, p.db, t);
    team_sum(s, p.team, buf, turn);
    const float a = s[0] * inv, mean = p.center ? s[1] * inv : 0.f;
    NormRow<T, VEC, PP> dx;
#pragma unroll
    for (int j = 0; j < PP; ++j) {
#pragma unroll
      for (int e = 0; e < VEC; ++e) d[j][e] = r * (fmaf(-n[j][e], a, d[j][e]) - mean);
      if constexpr (Z) {
        if (p.gate_first) {
          float gate[VEC], slope[VEC];
          norm_act<VEC>(p.act, zv[j], gate, slope);
#pragma unroll
          for (int e = 0; e < VEC; ++e) {
            slope[e] *= d[j][e] * raw[j][e];
            d[j][e] *= gate[e];
          }
          out.r[j].round(slope);
        }
      }
      dx.r[j].round(d[j]);
    }
    dx.store(p, m, p.y, p.ys, p.yb, t);
    if constexpr (Z)
      if (p.gate_first) out.store(p, m, p.dz, p.ds, p.db, t);
  }
  if (p.part == nullptr) return;
  // a column's sums over the block's teams that hold it, in their order
  const int teams = p.rows * p.span, each = p.team * PP * VEC;
  const int columns = p.shared ? p.W : p.D;
  const int groups = p.shared ? 1 : p.span, g0 = blockIdx.x % p.blocks_per_row * p.span;
  float *part = p.part +
                (int64_t)(p.shared ? blockIdx.x : blockIdx.x / p.blocks_per_row) * 2 * columns;
#pragma unroll
  for (int which = 0; which < 2; ++which) {
    __syncthreads();
    if (m.index < teams)
#pragma unroll
      for (int j = 0; j < PP; ++j)
#pragma unroll
        for (int e = 0; e < VEC; ++e)
          sums[m.index * each + (m.lane + j * p.team) * VEC + e] = which ? db[j][e] : dw[j][e];
    __syncthreads();
    for (int i = threadIdx.x; i < groups * p.W; i += blockDim.x) {
      const int q = i / p.W, c = i - q * p.W;
      if (!p.shared && g0 + q >= p.G) break;
      float v = 0.f;
      for (int k = q; k < teams; k += groups) v += sums[k * each + c];
      part[which * columns + (p.shared ? c : (g0 + q) * p.W + c)] = v;
    }
  }
}

// grid: columns of part (dweight's, then dbias's) in blocks of 32; 32 rows at a time.
__global__ void __launch_bounds__(1024) norm_sums_kernel(const float *part, int rows, int columns,
                                                         float *dw, float *db) {
  __shared__ float sums[32][33];
  const int c = blockIdx.x * 32 + threadIdx.x;
  float v = 0.f;
  if (c < 2 * columns)
    for (int r = threadIdx.y; r < rows; r += 32) v += part[(int64_t)r * 2 * columns + c];
  sums[threadIdx.y][threadIdx.x] = v;
  __syncthreads();
  if (threadIdx.y != 0 || c >= 2 * columns) return;
  for (int r = 1; r < 32; ++r) v += sums[r][threadIdx.x];
  if (c < columns) {
    if (dw) dw[c] = v;
  } else if (db) {
    db[c - columns] = v;
  }
}

}  // namespace

cudaError_t launch_norm_bwd(const NormParams &p, bool bf16, int vec, int pieces, int threads,
                            int blocks, cudaStream_t stream) {
  const int smem = p.part ? threads * pieces * vec * (int)sizeof(float) : 0;
  return norm_forms(bf16, vec, pieces, p.z != nullptr, [&](auto t, auto v, auto n, auto z) {
    using T = decltype(t);
    constexpr int VEC = decltype(v)::value, PP = decltype(n)::value;
    constexpr bool Z = decltype(z)::value;
    if (threads <= NORM_BWD_THREADS) {
      norm_bwd_kernel<T, VEC, PP, Z, false><<<blocks, threads, smem, stream>>>(p);
    } else {  // only with the most pieces a thread
      if constexpr (PP == norm_pieces(VEC))
        norm_bwd_kernel<T, VEC, PP, Z, true><<<blocks, threads, smem, stream>>>(p);
      else
        return cudaErrorInvalidConfiguration;
    }
    return cudaGetLastError();
  });
}

cudaError_t launch_norm_sums(const float *part, int rows, int columns, float *dw, float *db,
                             cudaStream_t stream) {
  norm_sums_kernel<<<(2 * columns + 31) / 32, dim3(32, 32), 0, stream>>>(part, rows, columns, dw, db);
  return cudaGetLastError();
}

}  // namespace gdn
