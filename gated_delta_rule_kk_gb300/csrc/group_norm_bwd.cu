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
#include "ptx.cuh"

namespace gdn {
namespace {

// Tokens on their way in the even kernels, in shared memory, each thread's pieces in places of
// its own (so that no thread waits for another): 36 KB a block and piece.  In registers there
// is room for two of them beside a token's values.  (2 x 4096 tokens of 16 heads of 128: 33.4 us,
// with two in registers 41.0, with four in shared memory 34.7, with three blocks an SM 43.)
constexpr int STAGES = 3;
constexpr int norm_bwd_ring(int pieces) { return STAGES * 3 * pieces * NORM_THREADS * 16; }

template <typename T, int VEC, int PP, NormGate GATE, int TEAM, bool WIDE>
__global__ void __launch_bounds__(norm_block(PP * VEC, WIDE), WIDE ? 1 : norm_bwd_per_sm(PP * VEC))
norm_bwd_kernel(NormParams p) {
  __shared__ float buf[2][NORM_WARPS][2];
  extern __shared__ __align__(16) float sums[];  // [threads][PP * VEC], or the ring
  const NormTeam<TEAM> m(p);
  if (!bounds_ok(p.team * p.rows * p.span <= (int)blockDim.x, p.err)) return;
  int turn = 0;
  const float inv = 1.f / (float)p.W;
  constexpr bool Z = GATE != NO_GATE, BEFORE = GATE == GATE_BEFORE;
  constexpr bool RING = TEAM != 0;
  constexpr int AHEAD = WIDE || RING ? 1 : norm_bwd_ahead(norm_words(sizeof(T), VEC, PP));
  float dw[PP][VEC], db[PP][VEC];
  NormCursor<T, TEAM> gc(p, m, p.dy, p.gs, p.gb, VEC), xc(p, m, p.x, p.xs, p.xb, VEC);
  NormCursor<T, TEAM> zc(p, m, p.z, p.zs, p.zb, VEC), dxc(p, m, p.y, p.ys, p.yb, VEC);
  NormCursor<T, TEAM> dzc(p, m, p.dz, p.ds, p.db, VEC);
  // (held where there is room: 51.3 -> 49.4 us; the forward gains nothing from it)
  const NormWeights<T, VEC, PP, PP * VEC <= 8> weight(p, m, p.weight), bias(p, m, p.bias);
  // dy, x and z of one of the next tokens: to the ring, and from it
  NormRow<T, VEC, PP> x[AHEAD], z[Z ? AHEAD : 1], g[AHEAD];
  auto place = [&](int stage, int which, int j) {
    return reinterpret_cast<T *>(sums) +
           (((stage * 3 + which) * PP + j) * NORM_THREADS + threadIdx.x) * VEC;
  };
  auto send = [&](int stage, int t) {
    const bool in = m.has(p, t);
    const T *from[3] = {gc.next(p, t), xc.next(p, t), Z ? zc.next(p, t) : nullptr};
    const void *any[3] = {p.dy, p.x, p.z};
#pragma unroll
    for (int which = 0; which < (Z ? 3 : 2); ++which)
#pragma unroll
      for (int j = 0; j < PP; ++j)
        ptx::cp_async16(place(stage, which, j), in ? from[which] + j * VEC * m.team(p) : any[which], in);
    ptx::cp_async_commit();
  };
  if constexpr (RING) {
#pragma unroll
    for (int i = 0; i < STAGES; ++i) send(i, m.t + i * p.step);
  } else {
#pragma unroll
    for (int i = 0; i < AHEAD; ++i) {
      const int t = m.t + i * p.step;
      const bool in = m.has(p, t);
      x[i].zero();
      g[i].zero();
      g[i].load(p, m, gc, t, in);
      x[i].load(p, m, xc, t, in);
      if constexpr (Z) {
        z[i].zero();
        z[i].load(p, m, zc, t, in);
      }
    }
  }
#pragma unroll
  for (int j = 0; j < PP; ++j)
#pragma unroll
    for (int e = 0; e < VEC; ++e) dw[j][e] = db[j][e] = 0.f;
  const int first = blockIdx.x / p.blocks_per_row * p.rows;
  for (int t0 = first, t = m.t, stage = 0; t0 < p.tokens; t0 += p.step, t += p.step) {
    const bool there = m.has(p, t);
    float n[PP][VEC], d[PP][VEC], gate[BEFORE ? PP : 1][VEC], slope[BEFORE ? PP : 1][VEC];
    if constexpr (RING) {
      ptx::cp_async_wait<STAGES - 1>();
#pragma unroll
      for (int j = 0; j < PP; ++j) {
        g[0].r[j].load(place(stage, 0, j));
        x[0].r[j].load(place(stage, 1, j));
        if constexpr (Z) z[0].r[j].load(place(stage, 2, j));
      }
    }
    // (what is wanted behind the root's sums stays as it lies in memory till then)
    const NormRow<T, VEC, PP> x_raw = x[0], g_raw = g[0], z_raw = z[0];
#pragma unroll
    for (int i = 1; i < AHEAD; ++i) {
      x[i - 1] = x[i];
      g[i - 1] = g[i];
      if constexpr (Z) z[i - 1] = z[i];
    }
#pragma unroll
    for (int j = 0; j < PP; ++j) {
      x_raw.r[j].widen(n[j]);
      if constexpr (BEFORE) {
        z_raw.r[j].widen(gate[j]);
        norm_act<VEC, true>(p.act, gate[j], gate[j], slope[j]);
        vmul<VEC>(n[j], n[j], gate[j]);
      }
    }
    if constexpr (RING) {
      send(stage, t + STAGES * p.step);
      stage = stage + 1 == STAGES ? 0 : stage + 1;
    } else {
      const int later = t + AHEAD * p.step;
      const bool more = m.has(p, later);
      g[AHEAD - 1].load(p, m, gc, later, more);
      x[AHEAD - 1].load(p, m, xc, later, more);
      if constexpr (Z) z[AHEAD - 1].load(p, m, zc, later, more);
    }
    const float r = norm_root<VEC, PP>(p, m, n, buf, turn);
    float dots[2] = {0.f, 0.f}, total[2] = {0.f, 0.f};  // of dn n and of dn
    NormRow<T, VEC, PP> out;
#pragma unroll
    for (int j = 0; j < PP; ++j) {
      vmul<VEC>(n[j], n[j], r);
      g_raw.r[j].widen(d[j]);
      float w[VEC], v[VEC];
      if (p.weight != nullptr) weight.get(p, m, j, w);
      if (GATE == GATE_AFTER || (!Z && p.act != GDN_ACT_NONE)) {  // m
        if (p.weight != nullptr) {
          vmul<VEC>(v, n[j], w);
        } else {
#pragma unroll
          for (int e = 0; e < VEC; ++e) v[e] = n[j][e];
        }
        if (p.bias != nullptr) {
          float b[VEC];
          bias.get(p, m, j, b);
          vadd<VEC>(v, v, b);
        }
        float by[VEC], gv[VEC];
        if constexpr (Z) {
          z_raw.r[j].widen(gv);
          norm_act<VEC, true>(p.act, gv, gv, by);
          vmul<VEC>(v, v, d[j]);
          vmul<VEC>(v, v, by);
          out.r[j].round(v);
          vmul<VEC>(d[j], d[j], gv);
        } else {
          norm_act<VEC, true>(p.act, v, v, by);
          vmul<VEC>(d[j], d[j], by);
        }
      }
      if (there) {
        vfma<VEC>(dw[j], d[j], n[j], dw[j]);
        vadd<VEC>(db[j], db[j], d[j]);
      }
      if (p.weight != nullptr) vmul<VEC>(d[j], d[j], w);
      vdot<VEC>(dots, d[j], n[j]);
      if (p.center) vsum<VEC>(total, d[j]);
    }
    if constexpr (GATE == GATE_AFTER) out.store(p, m, dzc, t, there);
    float s[2] = {dots[0] + dots[1], total[0] + total[1]};
    if (p.center) {
      team_sum(s, m.team(p), buf, turn);
    } else {
      float one[1] = {s[0]};
      team_sum(one, m.team(p), buf, turn);
      s[0] = one[0];
    }
    const float a = -s[0] * inv, mean = s[1] * inv;
    NormRow<T, VEC, PP> dx;
#pragma unroll
    for (int j = 0; j < PP; ++j) {
      vfma<VEC>(d[j], n[j], a, d[j]);
      if (p.center) vsub<VEC>(d[j], d[j], mean);
      vmul<VEC>(d[j], d[j], r);
      if constexpr (BEFORE) {
        float u[VEC];
        x_raw.r[j].widen(u);
        vmul<VEC>(u, u, d[j]);
        vmul<VEC>(u, u, slope[j]);
        out.r[j].round(u);
        vmul<VEC>(d[j], d[j], gate[j]);
      }
      dx.r[j].round(d[j]);
    }
    dx.store(p, m, dxc, t, there);
    if constexpr (BEFORE) out.store(p, m, dzc, t, there);
  }
  if constexpr (RING) ptx::cp_async_wait<0>();
  if (p.part == nullptr) return;
  // a column's sums over the block's teams that hold it, in their order
  const int teams = p.rows * p.span, each = m.team(p) * PP * VEC;
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
          sums[m.index * each + (m.lane + j * m.team(p)) * VEC + e] = which ? db[j][e] : dw[j][e];
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

// grid: columns of part (dweight's, then dbias's where wanted) in blocks of 32; a warp takes
// every 32nd row, then a column.
__global__ void __launch_bounds__(1024) norm_sums_kernel(const float *part, int rows, int columns,
                                                         float *dw, float *db) {
  __shared__ float sums[32][33];
  ptx::griddep_wait();  // launched while the kernel before it ends
  const int first = blockIdx.x * 32, lane = threadIdx.x, warp = threadIdx.y;
  float v = 0.f;
  if (first + lane < 2 * columns) {
    const float *at = part + first + lane;
#pragma unroll 8
    for (int r = warp; r < rows; r += 32) v += at[(int64_t)r * 2 * columns];
  }
  sums[warp][lane] = v;
  __syncthreads();
  v = sums[lane][warp];
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(~0u, v, o);
  const int c = first + warp;
  if (lane != 0 || c >= 2 * columns) return;
  if (c < columns) {
    if (dw) dw[c] = v;
  } else if (db) {
    db[c - columns] = v;
  }
}

}  // namespace

cudaError_t launch_norm_bwd(const NormParams &p, bool bf16, const NormPlan &plan, cudaStream_t stream) {
  const int sums = p.part ? plan.threads * plan.pieces * plan.vec * (int)sizeof(float) : 0;
  return norm_forms(bf16, plan, p, [&](auto t, auto v, auto n, auto gate, auto team) {
    using T = decltype(t);
    constexpr int VEC = decltype(v)::value, PP = decltype(n)::value;
    constexpr NormGate GATE = decltype(gate)::value;
    constexpr int TEAM = decltype(team)::value;
    if (plan.threads <= NORM_THREADS) {
      int smem = sums;
      if constexpr (TEAM != 0) {  // (the ring is more than the sums)
        smem = norm_bwd_ring(PP);
        const cudaError_t e = cudaFuncSetAttribute(norm_bwd_kernel<T, VEC, PP, GATE, TEAM, false>,
                                                   cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
        if (e != cudaSuccess) return e;
      }
      norm_bwd_kernel<T, VEC, PP, GATE, TEAM, false><<<plan.blocks, plan.threads, smem, stream>>>(p);
    } else {  // only with the most pieces a thread
      if constexpr (PP == norm_pieces(VEC))
        norm_bwd_kernel<T, VEC, PP, GATE, 0, true><<<plan.blocks, plan.threads, sums, stream>>>(p);
      else
        return cudaErrorInvalidConfiguration;
    }
    return cudaGetLastError();
  });
}

cudaError_t launch_norm_sums(const float *part, int rows, int columns, float *dw, float *db,
                             cudaStream_t stream) {
  const int wanted = db ? 2 * columns : columns;
  cudaLaunchAttribute early{};
  early.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  early.val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3((wanted + 31) / 32);
  cfg.blockDim = dim3(32, 32);
  cfg.stream = stream;
  cfg.attrs = &early;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, norm_sums_kernel, part, rows, columns, dw, db);
}

}  // namespace gdn
