// The inputs' gradients of the chunked gated delta rule on the tensor cores: what every chunk
// does by itself once its state h, the state's gradient D, and n and dr are there.
// delta_bwd.h has the formulas.
//
// A chunk and head reads 290 KB and writes 32 (K = V = 128), and multiplies
//   do h^T, dr h^T, n D^T [64][K] and do n^T, dr n^T [64][64],
// each over the V value columns, with h, D, n and dr as two bfloat16 pieces: 12.6 of the 15.2
// million multiplications of a chunk.  These five go to tcgen05, whose accumulators take all
// of tensor memory, while the warps finish the chunk before: they take over the accumulators
// (as fragments, which is how tcgen05.ld's 16x256b form gives them), apply gates and masks,
// and do what is left, dq += (dP L) k and dk += (dP L)^T q + .., on warp-level instructions.
// One block an SM, persistent, 20 warps: loads; the tcgen05 issuer; <h, D>; one that fetches
// q and k and adds up dbeta and dg; sixteen that finish.  (q and k come as a bulk copy a row:
// as 16-byte copies by all threads they held those up for 4500 cycles a chunk.)  Every wait is
// bounded; a warp whose wait ran out asks for nothing and arrives nowhere any more (a stage would
// be asked for before its copies have landed, which its barrier does not bear), so that the
// others' waits run out behind it.
// At 2 x 4096 tokens, 16 heads of 128, 135 us: 628 MB at 4.7 TB/s (69% of the copy rate), the
// tensor pipes busy 47% of the time; the finishing warps' phases, which wait for each other,
// set the pace.  (All on warp-level instructions, 16 warps a chunk, phase after phase: 245 us,
// of which the products took 6 of 18 us a chunk and waiting for loads 5.)
#include <algorithm>

#include "abi_check.h"
#include "delta_bwd_tc.cuh"

namespace gdn {
namespace {

constexpr int IN_WARPS = 20, IN_FINISH = 16;  // of a block; of them, the ones that finish

template <int KP>
struct InputsShared {
  static constexpr int PITCH = KP + 8, KQ = 2 * Q * PITCH * 2;  // q, k of an item
  static constexpr int DO_ = Q * VT * 2, ROWS = Block<KP>::ROWS, STATE = Block<KP>::STATE;
  // a value tile: do as 8 x 8 tiles [v][token] of tokens' rows, dr, n, h, D as they lie in the
  // workspace
  static constexpr int DR_AT = DO_, N_AT = DR_AT + ROWS, H_AT = N_AT + ROWS, D_AT = H_AT + STATE,
                       STAGE = D_AT + STATE;
  static constexpr int STAGES = 2 * KQ, MATS = STAGES + 2 * STAGE, SUMS = MATS + 2 * Block<KP>::SQUARE;
  // a head's sums by quarters of the columns or rows, and its gates; two sets, taken in turn
  static constexpr int SUM_SET = (4 * 6 + 1 + 5) * Q;
  static constexpr int BYTES = SUMS + 2 * SUM_SET * 4;
};

// Columns of tensor memory.
constexpr int XQ = 0, XK = 128, XS = 256, DP = 384, DA = 448;

// A chunk's place for the warps that finish it.
struct InputsItem {
  int64_t token;
  int len;
};

// The items of a block in turn: chunks x key heads, blockIdx.x, + gridDim.x, ..
struct InputsWalk {
  int64_t c, chunks;
  int hk, heads, dc, dh;
  __device__ __forceinline__ InputsWalk(int64_t chunks_, int heads_) : chunks(chunks_), heads(heads_) {
    c = blockIdx.x / heads;
    hk = blockIdx.x % heads;
    dc = gridDim.x / heads;
    dh = gridDim.x % heads;
  }
  __device__ __forceinline__ bool there() const { return c < chunks; }
  __device__ __forceinline__ void next() {
    c += dc;
    hk += dh;
    if (hk >= heads) {
      hk -= heads;
      ++c;
    }
  }
};

// N fragments (16 rows x 8 columns each) of this warp's quarter of tensor memory, rows 0 .. 15.
template <int N>
__device__ __forceinline__ void take_fragments(uint32_t at, float (*v)[4]) {
  static_assert(N == 2 || N == 4, "");
  uint32_t r[N * 4];
  if constexpr (N == 4)
    asm volatile(
        "tcgen05.ld.sync.aligned.16x256b.x4.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,"
        "%14,%15}, [%16];"
        : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]),
          "=r"(r[7]), "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]),
          "=r"(r[14]), "=r"(r[15])
        : "r"(at)
        : "memory");
  else
    asm volatile("tcgen05.ld.sync.aligned.16x256b.x2.b32 {%0,%1,%2,%3,%4,%5,%6,%7}, [%8];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]),
                   "=r"(r[6]), "=r"(r[7])
                 : "r"(at)
                 : "memory");
  asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory");
#pragma unroll
  for (int i = 0; i < N * 4; ++i) v[i / 4][i % 4] = __uint_as_float(r[i]);
}

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

__device__ __forceinline__ void finishers_meet() {
  asm volatile("bar.sync 1, %0;" ::"n"(32 * IN_FINISH) : "memory");
}

// A thread's part of a row [8 NT] of results (of each tile two neighbours, from 2 t) as
// bfloat16, where `in` and up to `most` columns: the row's four lanes exchange what they hold
// of four tiles, so that each writes 16 bytes of one.
template <int NT>
__device__ __forceinline__ void store_row(bf16 *to, const float (*v)[4], int e, int t, bool in,
                                          int most) {
  uint32_t w[NT];
#pragma unroll
  for (int j = 0; j < NT; ++j) {
    const __nv_bfloat162 h = __floats2bfloat162_rn(v[j][2 * e], v[j][2 * e + 1]);
    w[j] = *reinterpret_cast<const uint32_t *>(&h);
  }
  if constexpr (NT == 4) {
#pragma unroll
    for (int o = 1; o < 4; o <<= 1)
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        if (j & o) continue;  // lane t keeps its own side of words j and j + o
        const bool up = t & o;
        const uint32_t got = __shfl_xor_sync(~0u, up ? w[j] : w[j + o], o);
        if (up)
          w[j] = got;
        else
          w[j + o] = got;
      }
    if (in && 8 * t < most) *reinterpret_cast<uint4 *>(to + 8 * t) = make_uint4(w[0], w[1], w[2], w[3]);
  } else {
#pragma unroll
    for (int j = 0; j < NT; ++j)
      if (in && 8 * j < most) *reinterpret_cast<uint32_t *>(to + 8 * j + 2 * t) = w[j];
  }
}

// dr.v of a token whose beta is next to zero (dbeta is (dr.n) / beta of any other), by one warp.
template <int KP>
__device__ __forceinline__ float dot_value(const DeltaBwdParams &p, const Block<KP> &w, int64_t token,
                                           int head, int row) {
  const int lane = threadIdx.x & 31;
  float s = 0.f;
  for (int c = lane; c < p.V; c += 32) {
    const bf16 *dr = reinterpret_cast<const bf16 *>(w.dr(c / VT)) +
                     (c % VT / 8 * (Q / 8) + row / 8) * 64 + c % 8 * 8 + row % 8;
    s = fmaf(to_f32(dr[0]) + to_f32(dr[Q * VT]),
             to_f32(static_cast<const bf16 *>(p.v)[((token + row) * p.H + head) * p.V + c]), s);
  }
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) s += __shfl_xor_sync(~0u, s, o);
  return s;
}

// Items: chunks x key heads, a block's blockIdx.x, + gridDim.x, ..; the value heads of a key
// head follow one another, their dq and dk summed (GROUPED) in `scratch`, thread by thread.
template <int KP, bool GROUPED>
__global__ void __launch_bounds__(32 * IN_WARPS, 1) tc_inputs_kernel(DeltaBwdParams p) {
  using S = InputsShared<KP>;
  constexpr int NT = KP / 32, PITCH = S::PITCH;  // tiles of 8 columns of a warp's quarter of [64][KP]
  extern __shared__ __align__(128) unsigned char shared[];
  __shared__ uint64_t st_full[2], st_empty[2], x_full, x_empty, kq_full[2], pa_full, begun, summed[2], counted[2];
  __shared__ uint64_t through;
  __shared__ int pa_asked;
  __shared__ InputsItem place[2];
  __shared__ float hD[4];
  __shared__ uint32_t tmem_at;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int rep = p.H / p.Hg, tiles = (p.V + VT - 1) / VT;
  ptx::griddep_wait();
  const int64_t chunks = p.cu ? p.first[p.N] : p.chunks;  // (-1 with bad offsets)
  if (!bounds_ok(chunks <= p.chunks && gridDim.x <= DELTA_MAX_BLOCKS, p.err)) return;
  if (threadIdx.x == 0) {
    for (int s = 0; s < 2; ++s) {
      ptx::mbar_init(&st_full[s], 2);
      ptx::mbar_init(&st_empty[s], 2);
    }
    ptx::mbar_init(&x_full, 2);
    ptx::mbar_init(&x_empty, IN_FINISH);
    ptx::mbar_init(&pa_full, 1);
    ptx::mbar_init(&begun, 1);
    ptx::mbar_init(&through, 1);
    pa_asked = 0;
    for (int s = 0; s < 2; ++s) {
      ptx::mbar_init(&kq_full[s], 1);
      ptx::mbar_init(&summed[s], IN_FINISH);
      ptx::mbar_init(&counted[s], 1);
    }
    ptx::fence_mbar_init();
  }
  if (warp == 0) ptx::tmem_alloc<512>(&tmem_at);
  // (channels past K stay zero: the rows' copies end before them)
  for (int i = threadIdx.x; i < 2 * S::KQ / 16; i += 32 * IN_WARPS)
    reinterpret_cast<uint4 *>(shared)[i] = make_uint4(0, 0, 0, 0);
  ptx::fence_proxy_async_smem();
  ptx::tc_fence_before();
  __syncthreads();
  ptx::tc_fence_after();
  const uint32_t tmem = tmem_at;
  bool ok = true;
  // roles: finish; multiply and <h, D>; stages; the clerk
  const int role = warp == 0 ? 2 : warp < 3 ? 1 : warp == 3 ? 3 : 0;
  auto wait = [&](uint64_t *bar, int use) {
    ok = ptx::mbar_wait_bounded(bar, (uint32_t)(use & 1), ok ? ptx::role_polls(role) : 1u) && ok;
  };
  // for what was asked for and may still be on its way, whatever ran out
  auto settle = [&](uint64_t *bar, int use) {
    ok = ptx::mbar_wait_bounded(bar, (uint32_t)(use & 1), 1u << 22) && ok;
  };
  auto stage = [&](int s) { return shared + S::STAGES + (s & 1) * S::STAGE; };
  if (warp == 0) {  // stages: what the workspace has, and do's rows as a left operand of tcgen05
    int s = 0;
    for (InputsWalk it(chunks, p.Hg); it.there(); it.next()) {
      const DeltaChunk ch = delta_chunk(p, it.c);
      for (int head = it.hk * rep; head < (it.hk + 1) * rep; ++head) {
        const Block<KP> w(p, it.c, head);
        const bf16 *from = static_cast<const bf16 *>(p.dout) + (ch.token * p.H + head) * p.V;
        for (int v = 0; v < tiles; ++v, ++s) {
          if (s >= 2) wait(&st_empty[s & 1], s / 2 - 1);
          if (!__all_sync(~0u, ok)) break;
          unsigned char *to = stage(s);
          if (lane == 0)
            ptx::mbar_arrive_expect_tx(&st_full[s & 1], 2 * S::ROWS + 2 * S::STATE);
          __syncwarp();
          if (lane == 0) ptx::bulk_g2s(to + S::DR_AT, w.dr(v), S::ROWS, &st_full[s & 1]);
          if (lane == 1) ptx::bulk_g2s(to + S::N_AT, w.n(v), S::ROWS, &st_full[s & 1]);
          if (lane == 2) ptx::bulk_g2s(to + S::H_AT, w.h(v), S::STATE, &st_full[s & 1]);
          if (lane == 3) ptx::bulk_g2s(to + S::D_AT, w.D(v), S::STATE, &st_full[s & 1]);
          __syncwarp();
#pragma unroll
          for (int e = 0; e < 8; ++e) {  // four pieces of 8 rows at a time
            const int row = e * 8 + lane / 4, col = lane % 4, at = v * VT + col * 8;
            const bool in = row < ch.len && at < p.V;
            ptx::cp_async16(to + (col * 8 + row / 8) * 128 + row % 8 * 16,
                            in ? from + (int64_t)row * p.H * p.V + at : from, in);
          }
          ptx::cp_async_commit();
          ptx::cp_async_wait<0>();
          ptx::fence_proxy_async_smem();
          __syncwarp();
          if (lane == 0) ptx::mbar_arrive(&st_full[s & 1]);
        }
      }
    }
    // the last copies land before the warp ends, whoever else waits for them
    for (int k = max(0, s - 2); k < s; ++k) settle(&st_full[k & 1], k / 2);
  } else if (warp == 1) {  // the five products
    const uint32_t wide = ptx::idesc_bf16(64, KP, 0, 1), wide_t = ptx::idesc_bf16(64, KP, 1, 1);
    const uint32_t square = ptx::idesc_bf16(64, Q, 0, 1), square_t = ptx::idesc_bf16(64, Q, 1, 1);
    int m = 0, s = 0;  // heads and stages so far
    for (InputsWalk it(chunks, p.Hg); it.there(); it.next())
      for (int r = 0; r < rep; ++r, ++m) {
        if (m >= 1) wait(&x_empty, m - 1);
        ptx::tc_fence_after();
        for (int v = 0; v < tiles; ++v, ++s) {
          wait(&st_full[s & 1], s / 2);
          if (lane == 0 && ok) {
            ptx::tc_fence_after();
            unsigned char *at = stage(s);
#pragma unroll
            for (int kk = 0; kk < VT / 16; ++kk) {
              const uint32_t more = v > 0 || kk > 0;
              // 16 value columns are two rows of tiles
              auto rows = [&](int image, int piece) {
                return ptx::sdesc(at + image + piece * Q * VT * 2 + kk * 2048, 1024, 128);
              };
              auto state = [&](int image, int piece) {
                return ptx::sdesc(at + image + piece * KP * VT * 2 + kk * KP * 32, KP * 16, 128);
              };
              const uint64_t go = ptx::sdesc(at + kk * 2048, 1024, 128);
              const uint64_t dr = rows(S::DR_AT, 0), dl = rows(S::DR_AT, 1);
              const uint64_t n = rows(S::N_AT, 0), nl = rows(S::N_AT, 1);
              const uint64_t h = state(S::H_AT, 0), hl = state(S::H_AT, 1);
              const uint64_t D = state(S::D_AT, 0), Dl = state(S::D_AT, 1);
              ptx::mma_bf16(tmem + XQ, go, h, wide, more);
              ptx::mma_bf16(tmem + XK, dr, h, wide_t, more);
              ptx::mma_bf16(tmem + XS, n, D, wide_t, more);
              ptx::mma_bf16(tmem + DP, go, n, square, more);
              ptx::mma_bf16(tmem + DA, dr, n, square_t, more);
              ptx::mma_bf16(tmem + XQ, go, hl, wide, 1);
              ptx::mma_bf16(tmem + XK, dr, hl, wide_t, 1);
              ptx::mma_bf16(tmem + XS, n, Dl, wide_t, 1);
              ptx::mma_bf16(tmem + DP, go, nl, square, 1);
              ptx::mma_bf16(tmem + DA, dr, nl, square_t, 1);
              ptx::mma_bf16(tmem + XK, dl, h, wide_t, 1);
              ptx::mma_bf16(tmem + XS, nl, D, wide_t, 1);
              // (dg adds its products with k up over the chunk: without this 1.3e-5 off where V
              // is 8 or tokens are few, with it 6e-6; 2 us of 467)
              ptx::mma_bf16(tmem + XS, nl, Dl, wide_t, 1);
              ptx::mma_bf16(tmem + DA, dl, n, square_t, 1);
              // (its diagonal gives dbeta, of terms that cancel: without this 6.4e-6 off)
              ptx::mma_bf16(tmem + DA, dl, nl, square_t, 1);
            }
            ptx::mma_commit(&st_empty[s & 1]);
            if (v + 1 == tiles) ptx::mma_commit(&x_full);
          }
          __syncwarp();
        }
      }
    // no product is left on its way when tensor memory is given back
    if (lane == 0) ptx::mma_commit(&through);
    settle(&through, 0);
  } else if (warp == 2) {  // <h, D>
    int m = 0, s = 0;
    for (InputsWalk it(chunks, p.Hg); it.there(); it.next())
      for (int r = 0; r < rep; ++r, ++m) {
        float sum = 0.f;
        for (int v = 0; v < tiles; ++v, ++s) {
          wait(&st_full[s & 1], s / 2);
          const bf16 *h = reinterpret_cast<const bf16 *>(stage(s) + S::H_AT);
          const bf16 *D = reinterpret_cast<const bf16 *>(stage(s) + S::D_AT);
#pragma unroll 2
          for (int i = lane * 8; i < KP * VT; i += 256) {
            Row<bf16, 8> a[2], b[2];
            float x[2][8], y[2][8];
#pragma unroll
            for (int e = 0; e < 2; ++e) {
              a[e].load(h + e * KP * VT + i);
              b[e].load(D + e * KP * VT + i);
              a[e].widen(x[e]);
              b[e].widen(y[e]);
            }
            add_row<8>(x[0], x[0], x[1]);
            add_row<8>(y[0], y[0], y[1]);
#pragma unroll
            for (int e = 0; e < 8; ++e) sum = fmaf(x[0][e], y[0][e], sum);
          }
          __syncwarp();
          if (lane == 0 && ok) ptx::mbar_arrive(&st_empty[s & 1]);
        }
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(~0u, sum, o);
        // (with the accumulators taken over, x_full's phase before is over)
        if (m >= 1) wait(&x_empty, m - 1);
        if (lane == 0 && ok) {
          hD[m & 3] = sum;
          ptx::mbar_arrive(&x_full);
        }
      }
  } else if (warp == 3) {
    // The clerk: an item's q and k, one ahead of the item that is finished; of a finished head
    // dbeta, and dG summed from the end (lane l has tokens l and l + 32).
    int m = 0, n = 0;
    InputsWalk ahead(chunks, p.Hg);
    auto fetch = [&] {
      if (!ahead.there() || !__all_sync(~0u, ok)) return;
      const DeltaChunk ch = delta_chunk(p, ahead.c);
      bf16 *to = reinterpret_cast<bf16 *>(shared + (n & 1) * S::KQ);
      for (int row = ch.len; row < Q; ++row)  // (their weights are zero: they may not be NaN)
        for (int i = lane; i < PITCH / 8; i += 32) {
          reinterpret_cast<uint4 *>(to + row * PITCH)[i] = make_uint4(0, 0, 0, 0);
          reinterpret_cast<uint4 *>(to + (Q + row) * PITCH)[i] = make_uint4(0, 0, 0, 0);
        }
      ptx::fence_proxy_async_smem();
      if (lane == 0) place[n & 1] = {ch.token, ch.len};
      __syncwarp();
      if (lane == 0) ptx::mbar_arrive_expect_tx(&kq_full[n & 1], 2 * ch.len * p.K * 2);
      __syncwarp();
      const int64_t stride = (int64_t)p.Hg * p.K, from = ch.token * stride + ahead.hk * p.K;
      for (int row = lane; row < ch.len; row += 32) {
        ptx::bulk_g2s(to + row * PITCH, static_cast<const bf16 *>(p.q) + from + row * stride, p.K * 2,
                      &kq_full[n & 1]);
        ptx::bulk_g2s(to + (Q + row) * PITCH, static_cast<const bf16 *>(p.k) + from + row * stride,
                      p.K * 2, &kq_full[n & 1]);
      }
      ++n;
      ahead.next();
    };
    fetch();
    for (InputsWalk it(chunks, p.Hg); it.there(); it.next()) {
      const DeltaChunk ch = delta_chunk(p, it.c);
      for (int head = it.hk * rep; head < (it.hk + 1) * rep; ++head, ++m) {
        if (head == it.hk * rep) {
          wait(&begun, m / rep);  // the item before has read its q and k
          fetch();
        }
        wait(&summed[m & 1], m / 2);
        const float *sums = reinterpret_cast<const float *>(shared + S::SUMS) + (m & 1) * S::SUM_SET;
        const float *qd = sums, *kh = qd + 4 * Q, *kD = kh + 4 * Q, *rM = kD + 4 * Q, *rB = rM + 4 * Q;
        const float *cM = rB + 4 * Q, *rn = cM + 4 * Q, *beta = rn + 3 * Q, *eG = beta + Q;
        const float state = hD[m & 3];
        float d[2], db[2], kds[2], all = 0.f;
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          const int i = lane + 32 * e;
          auto all_of = [&](const float *x) { return (x[i] + x[Q + i]) + (x[2 * Q + i] + x[3 * Q + i]); };
          const float kd = all_of(kD), khi = all_of(kh);
          d[e] = all_of(rM) - all_of(cM) + all_of(qd) + beta[i] * khi;
          kds[e] = kd;
          if (p.g_is_cumsum) d[e] -= kd, all += kd;
          // dbeta = dr.n / beta, as n is beta times what it does not depend on it by (of a beta
          // next to nothing the products of dr's and n's pieces could fall below float32)
          const bool none = fabsf(beta[i]) < 1e-12f;
          db[e] = none ? khi + all_of(rB) : rn[i] / beta[i];
          for (unsigned z = __ballot_sync(~0u, none && i < ch.len); z; z &= z - 1) {
            const int l = __ffs(z) - 1;
            const float v = dot_value<KP>(p, Block<KP>(p, it.c, head), ch.token, head, l + 32 * e);
            if (lane == l) db[e] += v;
          }
          if (i < ch.len) p.dbeta[(ch.token + i) * p.H + head] = db[e];
        }
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) all += __shfl_xor_sync(~0u, all, o);
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
          delta_before(kds);
          d[0] += kds[0];
          d[1] += kds[1];
        }
#pragma unroll
        for (int e = 0; e < 2; ++e)
          if (lane + 32 * e < ch.len) p.dg[(ch.token + lane + 32 * e) * p.H + head] = d[e];
        __syncwarp();
        if (lane == 0 && ok) ptx::mbar_arrive(&counted[m & 1]);
      }
    }
    for (int k = max(0, n - 2); k < n; ++k) settle(&kq_full[k & 1], k / 2);  // all have landed
  } else {
    // Sixteen warps finish a head: rows 16 wm (their quarter of tensor memory), quarter wn of
    // the columns.
    const int tid = threadIdx.x - 128, wm = warp & 3, wn = (warp - 4) >> 2, g = lane >> 2, t = lane & 3;
    const uint32_t quarter = tmem + ((uint32_t)(32 * wm) << 16);
    bf16 *PL = reinterpret_cast<bf16 *>(shared + S::MATS), *AL = PL + 2 * Q * Q;
    int m = 0, n = 0;
    float gate = 0.f, less = 0.f;
    InputsWalk it(chunks, p.Hg);
    auto fetch_gates = [&](int64_t c, int head) {
      if (tid < 4 * Q) gate = Block<KP>(p, c, head).sc()[tid];
      if (tid < Q) less = Block<KP>(p, c, head).rest(tid);
    };
    if (it.there()) fetch_gates(it.c, it.hk * rep);
    for (; it.there(); ++n) {
      const int64_t c = it.c;
      const int hk = it.hk;
      it.next();  // (from here on the next one)
      wait(&kq_full[n & 1], n / 2);
      // (without its wait the place may be anything: no row is written)
      const int64_t token = place[n & 1].token;
      const int len = ok ? place[n & 1].len : 0;
      const bf16 *q = reinterpret_cast<const bf16 *>(shared + (n & 1) * S::KQ), *k = q + Q * PITCH;
      for (int head = hk * rep; head < (hk + 1) * rep; ++head, ++m) {
        // by quarters: q.dq_h, k.dk_h / beta, k.dk_s, rows of M, rows of B; columns of M by wm;
        // dr.n; gates and the sums' rests
        float *sums = reinterpret_cast<float *>(shared + S::SUMS) + (m & 1) * S::SUM_SET;
        float *qd = sums, *kh = qd + 4 * Q, *kD = kh + 4 * Q, *rM = kD + 4 * Q, *rB = rM + 4 * Q;
        float *cM = rB + 4 * Q, *rn = cM + 4 * Q, *sc = rn + Q;
        // (sums and rests side by side)
        const float2 *G = reinterpret_cast<const float2 *>(sc);
        const float *beta = sc + 2 * Q, *eG = sc + 3 * Q, *eR = sc + 4 * Q;
        const bool last = head + 1 == (hk + 1) * rep;
        if (m >= 2) wait(&counted[m & 1], m / 2 - 1);  // the sums' place is free
        if (tid < Q)
          reinterpret_cast<float2 *>(sc)[tid] = make_float2(gate, less);
        else if (tid < 4 * Q)
          sc[Q + tid] = gate;
        // the next head's gates, on their way meanwhile
        if (!last || it.there()) fetch_gates(last ? it.c : c, last ? it.hk * rep : head + 1);
        ptx::fence_proxy_async_smem();
        finishers_meet();
        if (tid == 0 && ok) {  // the head before is through: P and A to where dP L and dA L beta will be
          if (head == hk * rep) ptx::mbar_arrive(&begun);
          pa_asked = m + 1;
          ptx::mbar_arrive_expect_tx(&pa_full, 2 * Block<KP>::SQUARE);
          ptx::bulk_g2s(PL, Block<KP>(p, c, head).P(), 2 * Block<KP>::SQUARE, &pa_full);
        }
        wait(&x_full, m);
        ptx::tc_fence_after();
        float dq[NT][4], dk[NT][4], dP[2][4], dA[2][4];
        {
          float xs[NT][4];
          if (__all_sync(~0u, ok)) {
            take_fragments<NT>(quarter + XQ + wn * (KP / 4), dq);
            take_fragments<NT>(quarter + XK + wn * (KP / 4), dk);
            take_fragments<NT>(quarter + XS + wn * (KP / 4), xs);
            take_fragments<2>(quarter + DP + wn * 16, dP);
            take_fragments<2>(quarter + DA + wn * 16, dA);
          } else {  // products may be on their way
#pragma unroll
            for (int j = 0; j < NT; ++j)
#pragma unroll
              for (int e = 0; e < 4; ++e) {
                dq[j][e] = dk[j][e] = xs[j][e] = 0.f;
                if (j < 2) dP[j][e] = dA[j][e] = 0.f;
              }
          }
          ptx::tc_fence_before();
          __syncwarp();
          if (lane == 0 && ok) ptx::mbar_arrive(&x_empty);
          // the terms with h and D, and their products with q and k
          float a[2] = {}, b[2] = {}, d[2] = {};
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            const int row = 16 * wm + g + 8 * e;
            const float fq = p.scale * eG[row], fk = -eG[row], fs = eR[row], be = beta[row];
#pragma unroll
            for (int j = 0; j < NT; ++j) {
              const int at_ = at<PITCH>(row, wn * (KP / 4) + 8 * j + 2 * t);
              const float2 x = get_pair(q, at_), y = get_pair(k, at_);
#pragma unroll
              for (int u = 0; u < 2; ++u) {
                float &vq = dq[j][2 * e + u], &vk = dk[j][2 * e + u];
                const float ks = fs * xs[j][2 * e + u], yu = u ? y.y : y.x;
                vq *= fq;
                vk *= fk;
                a[e] = fmaf(vq, u ? x.y : x.x, a[e]);
                b[e] = fmaf(vk, yu, b[e]);
                d[e] = fmaf(ks, yu, d[e]);
                vk = fmaf(be, vk, ks);
              }
            }
          }
          put_rows(qd + wn * Q, 16 * wm + g, t, a[0], a[1]);
          put_rows(kh + wn * Q, 16 * wm + g, t, b[0], b[1]);
          put_rows(kD + wn * Q, 16 * wm + g, t, d[0], d[1]);
        }
        // M, dP L and dA L beta, each element of P and A replaced by the thread that read it
        wait(&pa_full, m);
        {
          float ms[2] = {}, bs[2] = {}, cols[2][2] = {};
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            const int row = 16 * wm + g + 8 * e;
            const float be = beta[row];
            const float2 Gr = G[row];
#pragma unroll
            for (int j = 0; j < 2; ++j) {
              const int col = 16 * wn + 8 * j + 2 * t;
              const int spot = at<64>(row, col);
              const float4 Gc = *reinterpret_cast<const float4 *>(G + col);
              const float2 Ph = get_pair(PL, spot), Pl = get_pair(PL + Q * Q, spot);
              const float2 Ah = get_pair(AL, spot), Al = get_pair(AL + Q * Q, spot);
              float pl[2], al[2];
#pragma unroll
              for (int u = 0; u < 2; ++u) {
                const float raw = dA[j][2 * e + u], own = dP[j][2 * e + u];
                if (row == col + u) rn[row] = raw;
                const bool in = row >= col + u && row < len, below = in && row > col + u;
                const float L = in ? __expf(delta_gap(Gr, u ? make_float2(Gc.z, Gc.w) : make_float2(Gc.x, Gc.y))) : 0.f;
                pl[u] = in ? L * p.scale * own : 0.f;
                al[u] = below ? -be * L * raw : 0.f;
                const float B = below ? -raw * (u ? Ah.y + Al.y : Ah.x + Al.x) : 0.f;
                const float M = fmaf(below ? own : 0.f, u ? Ph.y + Pl.y : Ph.x + Pl.x, be * B);
                ms[e] += M;
                bs[e] += B;
                cols[j][u] += M;
              }
              put_pair(PL, PL + Q * Q, spot, pl[0], pl[1]);
              put_pair(AL, AL + Q * Q, spot, al[0], al[1]);
            }
          }
          put_rows(rM + wn * Q, 16 * wm + g, t, ms[0], ms[1]);
          put_rows(rB + wn * Q, 16 * wm + g, t, bs[0], bs[1]);
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
        finishers_meet();
        // dq += PL k, dk += AL k + AL^T k + PL^T q; what is zero above or below is skipped
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          uint32_t a[4], al[4], b[NT / 2][4];
          auto add = [&](float (*to)[4], const bf16 *rows) {
#pragma unroll
            for (int u = 0; u < NT / 2; ++u) ldb_t<PITCH>(b[u], rows, wn * (KP / 4) + 16 * u, 16 * i);
#pragma unroll
            for (int u = 0; u < NT / 2; ++u) mma2(to + 2 * u, a, b[u]);
#pragma unroll
            for (int u = 0; u < NT / 2; ++u) mma2(to + 2 * u, al, b[u]);
          };
          if (i <= wm) {
            lda<64>(a, PL, 16 * wm, 16 * i);
            lda<64>(al, PL + Q * Q, 16 * wm, 16 * i);
            add(dq, k);
            lda<64>(a, AL, 16 * wm, 16 * i);
            lda<64>(al, AL + Q * Q, 16 * wm, 16 * i);
            add(dk, k);
          }
          if (i >= wm) {
            lda_t<64>(a, AL, 16 * wm, 16 * i);
            lda_t<64>(al, AL + Q * Q, 16 * wm, 16 * i);
            add(dk, k);
            lda_t<64>(a, PL, 16 * wm, 16 * i);
            lda_t<64>(al, PL + Q * Q, 16 * wm, 16 * i);
            add(dk, q);
          }
        }
        if (GROUPED) {
          float4 *total = reinterpret_cast<float4 *>(p.scratch) +
                          (int64_t)blockIdx.x * (Q * KP / 2) + tid;
#pragma unroll
          for (int j = 0; j < NT; ++j)
#pragma unroll
            for (int which = 0; which < 2; ++which) {
              float *x = which ? dk[j] : dq[j];
              float4 *at_ = total + (2 * j + which) * 32 * IN_FINISH;
              if (head > hk * rep) {
                const float4 y = *at_;
                x[0] += y.x; x[1] += y.y; x[2] += y.z; x[3] += y.w;
              }
              if (!last) *at_ = make_float4(x[0], x[1], x[2], x[3]);
            }
        }
        if (last) {
          bf16 *const to[2] = {static_cast<bf16 *>(p.dq), static_cast<bf16 *>(p.dk)};
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            const int row = 16 * wm + g + 8 * e;
#pragma unroll
            for (int which = 0; which < 2; ++which) {
              bf16 *out = to[which] + ((token + row) * p.Hg + hk) * p.K + wn * (KP / 4);
              store_row<NT>(out, which ? dk : dq, e, t, row < len, p.K - wn * (KP / 4));
            }
          }
        }
        __syncwarp();
        if (lane == 0 && ok) ptx::mbar_arrive(&summed[m & 1]);
      }
    }
  }
  if (threadIdx.x == 128 && pa_asked > 0) settle(&pa_full, pa_asked - 1);  // (that thread asked)
  if (!ok && lane == 0) record_error(p.err, GDN_ERR_TIMEOUT);
  ptx::tc_fence_before();
  __syncthreads();
  if (warp == 0) ptx::tmem_dealloc<512>(tmem);
}

template <int KP>
cudaError_t launch(const DeltaBwdParams &p, cudaStream_t stream) {
  const bool grouped = p.H > p.Hg;
  const void *kernel = grouped ? reinterpret_cast<const void *>(tc_inputs_kernel<KP, true>)
                               : reinterpret_cast<const void *>(tc_inputs_kernel<KP, false>);
  const cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                             InputsShared<KP>::BYTES);
  if (e != cudaSuccess) return e;
  const int64_t most = std::min<int64_t>(std::min(sm_count(), DELTA_MAX_BLOCKS), p.chunks * p.Hg);
  const unsigned blocks = (unsigned)most;
  return launch_behind(grouped ? tc_inputs_kernel<KP, true> : tc_inputs_kernel<KP, false>, dim3(blocks),
                       32 * IN_WARPS, InputsShared<KP>::BYTES, stream, p);
}

}  // namespace

cudaError_t launch_delta_inputs(const DeltaBwdParams &p, cudaStream_t stream) {
  return p.K <= 64 ? launch<64>(p, stream) : launch<128>(p, stream);
}

int64_t delta_bwd_tc_scratch(const DeltaBwdParams &p) {
  if (p.H == p.Hg) return 0;
  const int64_t blocks = std::min<int64_t>(DELTA_MAX_BLOCKS, p.chunks * p.Hg);
  return blocks * 2 * Q * (p.K <= 64 ? 64 : 128) * (int64_t)sizeof(float);
}

}  // namespace gdn
