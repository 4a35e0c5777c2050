// KDA for single tokens: T = 1..4 tokens of each request against a pool of states S [V, K],
//   S <- S diag(decay),  d = beta (v - S k),  S <- S + d k^T,  o = S q
// with q scaled, q and k of unit length, decay = exp(-e^A_log softplus(a + dt_bias)) per key
// channel and beta = sigmoid(b).
//
// A call is bound by the states, read and written once.  A thread holds four rows of a tile,
// one 16-byte piece of each (two above 128 float32 channels); both dot products are of the
// decayed state, S k and S q, so that they are summed over a row's lanes together, and
// o = S q + d (k . q).  A row's lanes hand sums on by halves: of a warp's rows each lane ends
// with one, works out its d and o, and hands d back.  The tokens of a call follow one another
// in registers, in float32; the state is rounded once: 4 T operations a state element.  (T tokens
// as one chunk, which the scalar gate's kernel takes, would be 3 T + 1: dots of the state as it
// was read with D_t k_t and D_t q_t, D_t the product of the decays up to t, the tokens' products
// with each other formed once a head.  Not tried.)
//
// 256 requests of 32 heads of 128 x 128, bf16 states: 99 us (547 MB at 5.5 TB/s, 81% of the copy
// rate); the ring's eight computing warps an SM issue on 69% of the cycles.  Four tokens: 214.
//
// What a head's rows share (decay, k, q of each token, v, beta, k . q) is formed once for an
// item, a warp a token (in the ring a warp an item), into shared memory.
#include <math.h>

#include <algorithm>

#include "abi_check.h"
#include "ptx.cuh"
#include "rows.cuh"

namespace gdn {
namespace {

struct KdParams {
  const void *q, *k, *v, *a, *b;
  const float *A_log, *dt_bias;
  void *state, *o;
  const int32_t *slots;
  int *err;
  int64_t qs, qb, ks, kb, vs, vb, as, ab, bs, bb, os, ob;
  int B, T, H, HV, K, V, pool;
  int l2norm, tok_f32, o_f32;
  float scale, eps;
  int vblocks, rows;          // tiles of a head, rows of a tile
  int stages;                 // of the ring
};

constexpr int KD_WARPS = 8, KD_ROWS = 4;
// The ring: two blocks an SM (three would leave a thread 48 registers, and its rows would
// spill), each with as many stages as its half of the shared memory holds, up to KD_STAGES.
// (A preparing warp skips the others' items; it may not skip a use of a barrier, so no more
// of them work than there are stages: 256 channels, one token or two, have five.)
constexpr int KD_STAGES = 6, KD_PREP = 4, KD_PER_SM = 2;
constexpr uint32_t KD_TILE = 16384;
// Shared memory of a ring, at most (the kernels' limit is this, whatever a call takes: calls
// of several threads set the same).
constexpr int KD_RING = 112 << 10;
constexpr int KD_THREADS = 32 * (KD_WARPS + KD_PREP + 2);

// A head's rows v .. end - 1 of one request.
struct KdItem {
  int b, h, v, end, slot;
};

// An item's coefficients (floats): decay, k and q [T][K], v [T][rows], beta and k . q [T], and
// whether its slot is good (so that the warps that take a tile need not look it up).
struct KdCoef {
  int K, R, T;
  __host__ __device__ KdCoef(int k, int r, int t) : K(k), R((r + 3) / 4 * 4), T(t) {}
  __host__ __device__ int decay(int t) const { return t * K; }
  __host__ __device__ int k(int t) const { return (T + t) * K; }
  __host__ __device__ int q(int t) const { return (2 * T + t) * K; }
  __host__ __device__ int v(int t) const { return 3 * T * K + t * R; }
  __host__ __device__ int beta(int t) const { return 3 * T * K + T * R + t; }
  __host__ __device__ int kq(int t) const { return 3 * T * K + T * R + T + t; }
  __host__ __device__ int good() const { return kq(T); }
  __host__ __device__ int bytes() const { return ((good() + 1) * 4 + 127) / 128 * 128; }
};

// One warp forms a token's coefficients: what it reads, and what it makes of it.  Lane l takes
// channels and rows l, l + 32, .., as many as the rows of LPR lanes and PP pieces can have.
template <typename S, int LPR, int PP>
struct KdToken {
  static constexpr int MOST = LPR * PP * 16 / (int)sizeof(S) / 32, ROWS = KD_WARPS * KD_ROWS / LPR;
  static_assert(MOST >= 1 && ROWS >= 1, "");
  float q[MOST], k[MOST], a[MOST], bias[MOST], v[ROWS], b, A_log;

  __device__ __forceinline__ void load(const KdParams &p, const KdItem &it, int t) {
    if (p.tok_f32)
      load_as<float>(p, it, t);
    else
      load_as<__nv_bfloat16>(p, it, t);
  }
  // Everything is asked for before anything is used: while states stream, a load takes some
  // microseconds.  (With the type looked at element by element they followed one another:
  // 120 us for 256 requests.)
  template <typename E>
  __device__ __forceinline__ void load_as(const KdParams &p, const KdItem &it, int t) {
    const int lane = threadIdx.x & 31, hk = it.h / (p.HV / p.H);
    const E *qat = static_cast<const E *>(p.q) + it.b * p.qb + t * p.qs + (int64_t)hk * p.K;
    const E *kat = static_cast<const E *>(p.k) + it.b * p.kb + t * p.ks + (int64_t)hk * p.K;
    const E *aat = static_cast<const E *>(p.a) + it.b * p.ab + t * p.as + (int64_t)it.h * p.K;
    const E *vat = static_cast<const E *>(p.v) + it.b * p.vb + t * p.vs + (int64_t)it.h * p.V + it.v;
    const float *bat = p.dt_bias ? p.dt_bias + (int64_t)it.h * p.K : nullptr;
    E rq[MOST], rk[MOST], ra[MOST], rv[ROWS];
#pragma unroll
    for (int i = 0; i < MOST; ++i) {
      const int ch = lane + 32 * i;
      const bool in = ch < p.K;  // (q and k of channels past K count in sums; the rest is not used)
      rq[i] = in ? qat[ch] : E(0.f);
      rk[i] = in ? kat[ch] : E(0.f);
      ra[i] = in ? aat[ch] : E(0.f);
      bias[i] = in && bat ? bat[ch] : 0.f;
    }
#pragma unroll
    for (int i = 0; i < ROWS; ++i)
      rv[i] = it.v + lane + 32 * i < it.end ? vat[lane + 32 * i] : E(0.f);
    const E rb = static_cast<const E *>(p.b)[it.b * p.bb + t * p.bs + it.h];
    A_log = p.A_log[it.h];
#pragma unroll
    for (int i = 0; i < MOST; ++i) {
      q[i] = to_f32(rq[i]);
      k[i] = to_f32(rk[i]);
      a[i] = to_f32(ra[i]);
    }
#pragma unroll
    for (int i = 0; i < ROWS; ++i) v[i] = to_f32(rv[i]);
    b = to_f32(rb);
  }

  __device__ __forceinline__ void put(const KdParams &p, const KdItem &it, int t, float *f) const {
    const int lane = threadIdx.x & 31;
    const KdCoef c(p.K, p.rows, p.T);
    float qq = 0.f, kk = 0.f, qk = 0.f;
#pragma unroll
    for (int i = 0; i < MOST; ++i) {
      qq = fmaf(q[i], q[i], qq);
      kk = fmaf(k[i], k[i], kk);
      qk = fmaf(q[i], k[i], qk);
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) {
      qq += __shfl_xor_sync(~0u, qq, o);
      kk += __shfl_xor_sync(~0u, kk, o);
      qk += __shfl_xor_sync(~0u, qk, o);
    }
    const float qn = p.l2norm ? p.scale / sqrtf(qq + p.eps) : p.scale;
    const float kn = p.l2norm ? 1.f / sqrtf(kk + p.eps) : 1.f;
    const float rate = -expf(A_log);
    float decay[MOST];  // side by side: each is a long chain
#pragma unroll
    for (int i = 0; i < MOST; ++i) {
      decay[i] = expf(rate * softplus(a[i] + bias[i]));
    }
#pragma unroll
    for (int i = 0; i < MOST; ++i) {
      const int ch = lane + 32 * i;
      if (ch >= p.K) continue;
      f[c.decay(t) + ch] = decay[i];
      f[c.k(t) + ch] = k[i] * kn;
      f[c.q(t) + ch] = q[i] * qn;
    }
#pragma unroll
    for (int i = 0; i < ROWS; ++i)
      if (it.v + lane + 32 * i < it.end) f[c.v(t) + lane + 32 * i] = v[i];
    if (lane == 0) {
      f[c.beta(t)] = 1.f / (1.f + expf(-b));
      f[c.kq(t)] = qk * qn * kn;
    }
  }
};

__device__ __forceinline__ void kd_put(const KdParams &p, const KdItem &it, int t, int r, float o) {
  const int64_t at = it.b * p.ob + t * p.os + (int64_t)it.h * p.V + r;
  if (p.o_f32)
    static_cast<float *>(p.o)[at] = o;
  else
    static_cast<__nv_bfloat16 *>(p.o)[at] = __float2bfloat16_rn(o);
}

// Sums of KD_ROWS rows over their LPR lanes; each lane is left with one row's.
template <int LPR>
__device__ __forceinline__ float kd_row_sums(float (&v)[KD_ROWS]) {
  const int lane = threadIdx.x & 31;
#pragma unroll
  for (int n = KD_ROWS / 2, o = LPR / 2; o > 0; n /= 2, o /= 2) {
    if (n > 0) {
      const bool up = lane & o;
#pragma unroll
      for (int j = 0; j < n; ++j) {
        const float send = up ? v[j] : v[j + n], keep = up ? v[j + n] : v[j];
        v[j] = keep + __shfl_xor_sync(~0u, send, o);
      }
    } else {
      v[0] += __shfl_xor_sync(~0u, v[0], o);
    }
  }
  return v[0];
}

// A thread's pieces of a tile: rows warp_row + lane / LPR + j 32 / LPR, channels
// (lane % LPR + i LPR) VEC.
template <typename S, int LPR, int PP>
struct KdTile {
  static constexpr int VEC = 16 / (int)sizeof(S), RPS = 32 / LPR;
  Row<S, VEC> raw[KD_ROWS][PP];

  static __device__ __forceinline__ int row(int j) { return (threadIdx.x & 31) / LPR + j * RPS; }
  static __device__ __forceinline__ int channel(int i) {
    return ((threadIdx.x & 31) % LPR + i * LPR) * VEC;
  }

  __device__ __forceinline__ void load(const S *tile, int first, int rows, int K) {
#pragma unroll
    for (int j = 0; j < KD_ROWS; ++j)
#pragma unroll
      for (int i = 0; i < PP; ++i) {
        if (first + row(j) < rows && channel(i) < K)
          raw[j][i].load(tile + (int64_t)(first + row(j)) * K + channel(i));
        else
          raw[j][i].zero();
      }
  }

  // The call's tokens on the rows, back to `tile`.
  template <int TM>
  __device__ __forceinline__ void take(const KdParams &p, const KdItem &it, S *tile, int first,
                                       const float *f) {
    const int lane = threadIdx.x & 31, rows = it.end - it.v, K = p.K;
    const KdCoef c(K, p.rows, p.T);
    // of the rows of its group of LPR lanes, a lane is left with row `mine`
    const int mine = (lane % LPR) / (LPR / KD_ROWS), own = first + row(mine);
    const bool writes = lane % (LPR / KD_ROWS) == 0 && own < rows;
    float s[KD_ROWS][PP][VEC];
#pragma unroll
    for (int j = 0; j < KD_ROWS; ++j)
#pragma unroll
      for (int i = 0; i < PP; ++i) raw[j][i].widen(s[j][i]);
#pragma unroll
    for (int t = 0; t < TM; ++t) {
      if (t >= p.T) break;
      float sk[KD_ROWS], sq[KD_ROWS], kv[PP][VEC];
#pragma unroll
      for (int j = 0; j < KD_ROWS; ++j) sk[j] = sq[j] = 0.f;
#pragma unroll
      for (int i = 0; i < PP; ++i) {
        float dv[VEC], qv[VEC];
#pragma unroll
        for (int e = 0; e < VEC; e += 4) {
          float4 x = make_float4(0.f, 0.f, 0.f, 0.f), y = x, z = x;
          if (channel(i) < K) {
            x = *reinterpret_cast<const float4 *>(f + c.decay(t) + channel(i) + e);
            y = *reinterpret_cast<const float4 *>(f + c.k(t) + channel(i) + e);
            z = *reinterpret_cast<const float4 *>(f + c.q(t) + channel(i) + e);
          }
          dv[e] = x.x; dv[e + 1] = x.y; dv[e + 2] = x.z; dv[e + 3] = x.w;
          kv[i][e] = y.x; kv[i][e + 1] = y.y; kv[i][e + 2] = y.z; kv[i][e + 3] = y.w;
          qv[e] = z.x; qv[e + 1] = z.y; qv[e + 2] = z.z; qv[e + 3] = z.w;
        }
#pragma unroll
        for (int j = 0; j < KD_ROWS; ++j) {
          float a[2] = {0.f, 0.f}, b[2] = {0.f, 0.f};
          mul_row<VEC>(s[j][i], s[j][i], dv);
#pragma unroll
          for (int e = 0; e < VEC; e += 2) {
            fma_row<2>(a, s[j][i] + e, kv[i] + e);
            fma_row<2>(b, s[j][i] + e, qv + e);
          }
          sk[j] += a[0] + a[1];
          sq[j] += b[0] + b[1];
        }
      }
      const float pred = kd_row_sums<LPR>(sk), out = kd_row_sums<LPR>(sq);
      const float v = own < rows ? f[c.v(t) + own] : 0.f;
      const float d = f[c.beta(t)] * (v - pred);
      if (writes) kd_put(p, it, t, it.v + own, fmaf(d, f[c.kq(t)], out));
#pragma unroll
      for (int j = 0; j < KD_ROWS; ++j) {
        const float dj = __shfl_sync(~0u, d, lane / LPR * LPR + j * (LPR / KD_ROWS));
        const float dd[2] = {dj, dj};
#pragma unroll
        for (int i = 0; i < PP; ++i)
#pragma unroll
          for (int e = 0; e < VEC; e += 2) fma_row<2>(s[j][i] + e, dd, kv[i] + e);
      }
    }
#pragma unroll
    for (int j = 0; j < KD_ROWS; ++j)
#pragma unroll
      for (int i = 0; i < PP; ++i) {
        if (first + row(j) >= rows || channel(i) >= K) continue;
        raw[j][i].round(s[j][i]);
        raw[j][i].store(tile + (int64_t)(first + row(j)) * K + channel(i));
      }
  }
};

template <typename S>
__device__ __forceinline__ S *kd_tile_at(const KdParams &p, const KdItem &it) {
  return static_cast<S *>(p.state) + (((int64_t)it.slot * p.HV + it.h) * p.V + it.v) * p.K;
}

// Items in turn, i, i + step, ..: the divisions are done once (each of an item's warps doing
// them anew took most of the ring's instructions).
struct KdWalk {
  int b, h, v, db, dh, dv;  // request, head, tile; and the step's
  __device__ __forceinline__ KdWalk(const KdParams &p, unsigned i, unsigned step) {
    const unsigned heads = p.HV, tiles = p.vblocks;
    v = i % tiles;
    h = i / tiles % heads;
    b = i / tiles / heads;
    dv = step % tiles;
    dh = step / tiles % heads;
    db = step / tiles / heads;
  }
  __device__ __forceinline__ void next(const KdParams &p) {
    v += dv;
    h += dh;
    b += db;
    if (v >= p.vblocks) {
      v -= p.vblocks;
      ++h;
    }
    if (h >= p.HV) {
      h -= p.HV;
      ++b;
    }
  }
  __device__ __forceinline__ KdItem place(const KdParams &p) const {  // all but its slot
    KdItem it;
    it.v = v * p.rows;
    it.end = min(it.v + p.rows, p.V);
    it.b = b;
    it.h = h;
    it.slot = 0;
    return it;
  }
  __device__ __forceinline__ KdItem item(const KdParams &p) const {
    KdItem it = place(p);
    it.slot = p.slots ? p.slots[b] : b;
    return it;
  }
};

__device__ __forceinline__ bool kd_good(const KdParams &p, const KdItem &it) {
  return it.slot >= 0 && it.slot < p.pool;
}

// Zeros for the tokens of a request whose slot is bad; threads 0 .. n - 1 take part.
__device__ __forceinline__ void kd_refuse(const KdParams &p, const KdItem &it, int tid, int n) {
  if (tid == 0) record_error(p.err, GDN_ERR_BAD_SLOT);
  for (int t = 0; t < p.T; ++t)
    for (int r = it.v + tid; r < it.end; r += n) kd_put(p, it, t, r, 0.f);
}

// Few states, or several tokens: one block a tile.  The rows are on their way while the coefficients form.
template <typename S, int LPR, int PP, int TM>
__global__ void __launch_bounds__(32 * KD_WARPS) kda_decode_kernel(KdParams p) {
  extern __shared__ __align__(128) float coef[];
  constexpr int WARP_ROWS = KD_ROWS * 32 / LPR;
  const int warp = threadIdx.x >> 5;
  const KdItem it = KdWalk(p, blockIdx.x, 1).item(p);
  if (!bounds_ok(it.b < p.B && it.h < p.HV && it.v < p.V && p.rows <= KD_WARPS * WARP_ROWS, p.err))
    return;
  if (!kd_good(p, it)) return kd_refuse(p, it, threadIdx.x, blockDim.x);
  S *tile = kd_tile_at<S>(p, it);
  KdTile<S, LPR, PP> rows;
  rows.load(tile, warp * WARP_ROWS, it.end - it.v, p.K);
  if (warp < p.T) {
    KdToken<S, LPR, PP> token;
    token.load(p, it, warp);
    token.put(p, it, warp, coef);
  }
  __syncthreads();
  rows.template take<TM>(p, it, tile, warp * WARP_ROWS, coef);
}

// Many states of one token (float32 ones of two) stream through a ring of bulk copies: `stages` tiles, each with its item's
// coefficients beside it.  Warps: KD_WARPS that take the tiles in place, KD_PREP that form
// the coefficients (every KD_PREP-th item each), one that loads and one that stores tiles.
// Every wait is bounded.  A warp whose wait ran out leaves: it touches no stage and arrives
// nowhere any more, so that the others' waits run out behind it.  (An arrival without its wait
// would let a stage be asked for before its copy has landed, which its barrier does not bear, or
// be stored before it is done.)  A state is the call's then, or as it was.
template <typename S, int LPR, int PP, int TM>
__global__ void __launch_bounds__(KD_THREADS, KD_PER_SM)
kda_decode_ring_kernel(KdParams p, int items) {
  extern __shared__ __align__(128) unsigned char ring[];
  __shared__ uint64_t full[KD_STAGES], ready[KD_STAGES], done[KD_STAGES], empty[KD_STAGES];
  constexpr int WARP_ROWS = KD_ROWS * 32 / LPR;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int role = warp < KD_WARPS ? 0 : warp < KD_WARPS + KD_PREP ? 1 : warp - KD_WARPS - KD_PREP + 2;
  const int coef_bytes = KdCoef(p.K, p.rows, p.T).bytes(), stages = p.stages;
  if (tid == 0) {
    for (int s = 0; s < stages; ++s) {
      ptx::mbar_init(&full[s], 1);
      ptx::mbar_init(&ready[s], 1);
      ptx::mbar_init(&done[s], KD_WARPS);
      ptx::mbar_init(&empty[s], 1);
    }
    ptx::fence_mbar_init();
  }
  __syncthreads();
  if (!bounds_ok(stages >= KD_PREP && stages <= KD_STAGES && p.rows > 0 &&
                     p.rows <= KD_WARPS * WARP_ROWS &&
                     p.rows * p.K * (int)sizeof(S) <= (int)KD_TILE,
                 p.err))
    return;
  bool ok = true;
  auto wait = [&](uint64_t *bar, int use) {
    ok = ptx::mbar_wait_bounded(bar, (uint32_t)(use & 1), ok ? ptx::role_polls(role) : 1u) && ok;
  };
  auto bytes_of = [&](const KdItem &it) {
    return (uint32_t)((it.end - it.v) * p.K * (int)sizeof(S));
  };
  auto coef = [&](int s) {
    return reinterpret_cast<float *>(ring + stages * KD_TILE + s * coef_bytes);
  };
  int n = 0;  // items of this block so far
  KdWalk walk(p, blockIdx.x, gridDim.x);
  if (warp < KD_WARPS) {
    for (int i = blockIdx.x; i < items; i += gridDim.x, ++n, walk.next(p)) {
      const int s = n % stages;
      const KdItem it = walk.place(p);
      wait(&ready[s], n / stages);
      wait(&full[s], n / stages);
      if (!__all_sync(~0u, ok)) break;
      if (coef(s)[KdCoef(p.K, p.rows, p.T).good()] != 0.f) {
        if (warp * WARP_ROWS < it.end - it.v) {
          S *tile = reinterpret_cast<S *>(ring + s * KD_TILE);
          KdTile<S, LPR, PP> rows;
          rows.load(tile, warp * WARP_ROWS, it.end - it.v, p.K);
          rows.template take<TM>(p, it, tile, warp * WARP_ROWS, coef(s));
        }
      } else {
        kd_refuse(p, it, tid, 32 * KD_WARPS);
      }
      ptx::fence_proxy_async_smem();
      __syncwarp();
      if (lane == 0) ptx::mbar_arrive(&done[s]);
    }
  } else if (warp < KD_WARPS + KD_PREP) {
    for (int i = blockIdx.x; i < items; i += gridDim.x, ++n, walk.next(p)) {
      if (n % KD_PREP != warp - KD_WARPS) continue;
      const int s = n % stages;
      const KdItem it = walk.item(p);
      KdToken<S, LPR, PP> token;
      token.load(p, it, 0);
      if (n >= stages) wait(&done[s], n / stages - 1);
      if (!__all_sync(~0u, ok)) break;
      token.put(p, it, 0, coef(s));
      for (int t = 1; t < p.T; ++t) {
        token.load(p, it, t);
        token.put(p, it, t, coef(s));
      }
      if (lane == 0) coef(s)[KdCoef(p.K, p.rows, p.T).good()] = kd_good(p, it) ? 1.f : 0.f;
      __syncwarp();
      if (lane == 0) ptx::mbar_arrive(&ready[s]);
    }
  } else if (warp == KD_WARPS + KD_PREP) {
    for (int i = blockIdx.x; i < items; i += gridDim.x, ++n, walk.next(p)) {
      const int s = n % stages;
      const KdItem it = walk.item(p);
      if (n >= stages) wait(&empty[s], n / stages - 1);
      if (!__all_sync(~0u, ok)) break;
      if (lane == 0) {
        if (kd_good(p, it)) {
          ptx::mbar_arrive_expect_tx(&full[s], bytes_of(it));
          ptx::bulk_g2s(ring + s * KD_TILE, kd_tile_at<S>(p, it), bytes_of(it), &full[s]);
        } else {
          ptx::mbar_arrive(&full[s]);
        }
      }
      __syncwarp();
    }
    // the last copies land before the warp ends, whoever else waits for them
    for (int k = max(0, n - stages); k < n; ++k)
      ok = ptx::mbar_wait_bounded(&full[k % stages], (uint32_t)(k / stages & 1), 1u << 22) && ok;
  } else {
    for (int i = blockIdx.x; i < items; i += gridDim.x, ++n, walk.next(p)) {
      const int s = n % stages;
      const KdItem it = walk.item(p);
      wait(&done[s], n / stages);
      if (!__all_sync(~0u, ok)) break;
      if (lane == 0) {
        if (kd_good(p, it)) ptx::bulk_s2g(kd_tile_at<S>(p, it), ring + s * KD_TILE, bytes_of(it));
        ptx::bulk_commit();
        if (n > 0) {  // the store before has read its tile
          ptx::bulk_wait_read<1>();
          ptx::mbar_arrive(&empty[(n - 1) % stages]);
        }
      }
      __syncwarp();
    }
    if (lane == 0) ptx::bulk_wait<0>();
  }
  if (!ok && lane == 0) record_error(p.err, GDN_ERR_TIMEOUT);
}

// Tiles a block of the ring from where it is the faster one; 0: nowhere.  Its warps form tokens'
// coefficients for several tiles in turn and are what a call of several tokens waits for; the
// direct kernel has a warp a token.  Requests of 32 heads of 128 x 128, ring / direct, us:
//   bf16 states  1 token: 8 requests (1.7 tiles a block) 7.5 / 7.0, 16 9.9 / 10.7, 64 27.8 / 33.9,
//                256 97.6 / 138.8; 2 tokens: 16 14.2 / 12.3, 256 161.6 / 161.0;
//                4 tokens: 2 12.0 / 4.9, 256 285 / 214
//   float32      1 token: 8 (3.4) 8.5 / 7.6, 16 (6.7) 12.6 / 13.3, 256 169.5 / 197;
//                2 tokens: 16 17.5 / 15.8, 64 (27) 57.7 / 61.4, 256 205.8 / 228.8;
//                4 tokens: 3 12.3 / 6.2, 256 363 / 302
template <typename S, int TM>
constexpr int kd_ring_from() {
  return TM == 1 ? 4 : TM == 2 && sizeof(S) == 4 ? 16 : 0;
}

template <typename S, int LPR, int PP, int TM>
cudaError_t launch_kda(KdParams &p, cudaStream_t stream) {
  constexpr int ROWS = KD_WARPS * KD_ROWS * 32 / LPR;
  const int64_t bh = (int64_t)p.B * p.HV;
  const int rows = std::min(ROWS, (int)(KD_TILE / (p.K * sizeof(S))));
  p.vblocks = (p.V + rows - 1) / rows;
  p.rows = (p.V + p.vblocks - 1) / p.vblocks;
  const int coef = KdCoef(p.K, p.rows, p.T).bytes();
  const int64_t items = bh * p.vblocks;
  if constexpr (kd_ring_from<S, TM>() > 0) {
    const int blocks = KD_PER_SM * sm_count();
    if (items >= kd_ring_from<S, TM>() * blocks && items <= 0x7fff0000) {
      p.stages = std::min(KD_STAGES, KD_RING / ((int)KD_TILE + coef));
      const int smem = p.stages * ((int)KD_TILE + coef);
      const cudaError_t e = cudaFuncSetAttribute(kda_decode_ring_kernel<S, LPR, PP, TM>,
                                                 cudaFuncAttributeMaxDynamicSharedMemorySize, KD_RING);
      if (e != cudaSuccess) return e;
      kda_decode_ring_kernel<S, LPR, PP, TM><<<blocks, KD_THREADS, smem, stream>>>(p, (int)items);
      return cudaGetLastError();
    }
  }
  kda_decode_kernel<S, LPR, PP, TM><<<(unsigned)items, 32 * KD_WARPS, coef, stream>>>(p);
  return cudaGetLastError();
}

template <typename S, int LPR, int PP>
cudaError_t launch_tokens(KdParams &p, cudaStream_t stream) {
  if (p.T == 1) return launch_kda<S, LPR, PP, 1>(p, stream);
  if (p.T == 2) return launch_kda<S, LPR, PP, 2>(p, stream);
  return launch_kda<S, LPR, PP, 4>(p, stream);
}

template <typename S>
cudaError_t launch_pieces(KdParams &p, cudaStream_t stream) {
  const int pieces = p.K * (int)sizeof(S) / 16;
  if (pieces <= 8) return launch_tokens<S, 8, 1>(p, stream);
  if (pieces <= 16) return launch_tokens<S, 16, 1>(p, stream);
  if constexpr (sizeof(S) == 4)
    if (pieces > 32) return launch_tokens<S, 32, 2>(p, stream);
  return launch_tokens<S, 32, 1>(p, stream);
}

}  // namespace
}  // namespace gdn

using namespace gdn;

extern "C" gdn_status_t kda_decode(const kda_decode_args *args, gdn_stream_t stream) {
  (void)set_host_error(GDN_OK, "");
  CHECK_THAT(args != nullptr, GDN_ERR_INVALID_ARG, "args is NULL");
  const kda_decode_args &a = *args;
  CHECK_DTYPE(a.dtype, "dtype");
  CHECK_DTYPE(a.state_dtype, "state_dtype");
  CHECK_THAT(a.B >= 1 && a.H >= 1 && a.HV >= 1 && a.K >= 1 && a.V >= 1, GDN_ERR_INVALID_ARG,
             "sizes must be positive (B=%d heads=%d/%d K=%d V=%d)", a.B, a.H, a.HV, a.K, a.V);
  CHECK_THAT(a.T >= 1 && a.T <= 4, GDN_ERR_UNSUPPORTED, "T must be 1..4 (got %d)", a.T);
  CHECK_THAT(a.HV % a.H == 0, GDN_ERR_UNSUPPORTED, "HV (%d) must be a multiple of H (%d)", a.HV, a.H);
  CHECK_THAT(a.HV <= MAX_GRID_YZ, GDN_ERR_UNSUPPORTED, "HV (%d) must be at most %d", a.HV, MAX_GRID_YZ);
  CHECK_THAT(a.K % 8 == 0 && a.K <= 256, GDN_ERR_UNSUPPORTED,
             "K (%d) must be a multiple of 8 up to 256", a.K);
  CHECK_THAT(a.V <= MAX_TOKENS, GDN_ERR_UNSUPPORTED, "V (%d) must be at most %d", a.V, MAX_TOKENS);
  CHECK_THAT(a.pool >= 1, GDN_ERR_INVALID_ARG, "pool must be positive (got %d)", a.pool);
  CHECK_THAT(a.slot_indices != nullptr || a.pool >= a.B, GDN_ERR_INVALID_ARG,
             "identity slots need pool (%d) >= B (%d)", a.pool, a.B);
  CHECK_FLAG(a.use_qk_l2norm, "use_qk_l2norm");
  CHECK_FLAG(a.o_fp32, "o_fp32");
  CHECK_THAT(isfinite(a.scale) && isfinite(a.eps), GDN_ERR_INVALID_ARG, "scale and eps must be finite");
  CHECK_TOKENS(a.q, "q", a.dtype);
  CHECK_TOKENS(a.k, "k", a.dtype);
  CHECK_TOKENS(a.v, "v", a.dtype);
  CHECK_TOKENS(a.a, "a", a.dtype);
  CHECK_TOKENS(a.b, "b", a.dtype);
  CHECK_TOKENS(a.o, "o", a.o_fp32 ? GDN_F32 : a.dtype);
  CHECK_PTR(a.A_log, "A_log");
  CHECK_OPT_PTR(a.dt_bias, "dt_bias");
  CHECK_PTR(a.state, "state");
  CHECK_OPT_PTR(a.slot_indices, "slot_indices");
  const int64_t hk = (int64_t)a.H * a.K, hv = (int64_t)a.HV * a.V, ha = (int64_t)a.HV * a.K;
  CHECK_THAT(a.q_stride >= hk && a.k_stride >= hk && a.v_stride >= hv && a.a_stride >= ha &&
                 a.b_stride >= a.HV && a.o_stride >= hv,
             GDN_ERR_INVALID_ARG, "a token stride is less than its row");
  CHECK_THAT((int64_t)a.B * a.HV * (((int64_t)a.V + 7) / 8) <= 0x7fffffff, GDN_ERR_UNSUPPORTED,
             "B * HV * V (%d * %d * %d) is too large for one call", a.B, a.HV, a.V);
  KdParams p{};
  const bool many = a.B > 1, tokens = a.T > 1;
  p.q = a.q; p.k = a.k; p.v = a.v; p.a = a.a; p.b = a.b; p.o = a.o;
  p.A_log = a.A_log; p.dt_bias = a.dt_bias; p.state = a.state; p.slots = a.slot_indices;
  p.qs = tokens ? a.q_stride : 0; p.qb = many ? a.q_batch_stride : 0;
  p.ks = tokens ? a.k_stride : 0; p.kb = many ? a.k_batch_stride : 0;
  p.vs = tokens ? a.v_stride : 0; p.vb = many ? a.v_batch_stride : 0;
  p.as = tokens ? a.a_stride : 0; p.ab = many ? a.a_batch_stride : 0;
  p.bs = tokens ? a.b_stride : 0; p.bb = many ? a.b_batch_stride : 0;
  p.os = tokens ? a.o_stride : 0; p.ob = many ? a.o_batch_stride : 0;
  p.B = a.B; p.T = a.T; p.H = a.H; p.HV = a.HV; p.K = a.K; p.V = a.V; p.pool = a.pool;
  p.l2norm = a.use_qk_l2norm;
  p.tok_f32 = a.dtype == GDN_F32;
  p.o_f32 = a.o_fp32 || a.dtype == GDN_F32;
  p.scale = a.scale > 0.f ? a.scale : 1.f / sqrtf((float)a.K);
  p.eps = a.eps >= 0.f ? a.eps : 1e-6f;
  p.err = device_error_word();
  if (p.err == nullptr) return launch_status(cudaGetLastError(), "device error word");
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  return launch_status(a.state_dtype == GDN_BF16 ? launch_pieces<__nv_bfloat16>(p, s)
                                                 : launch_pieces<float>(p, s),
                       "KDA token launch");
}
