// The states of the chunked gated delta rule forward and their gradients backward, a chunk
// after another, for the gradient on the tensor cores.
//
// What bounds a walk is the way from one state to the next, three products that wait for one
// another; there are only as many walks as heads, sequences and value columns give.  Two warps
// carry 16 value columns.  They hold the state transposed, S [16][K], in their accumulators,
// half of the channels each, and as an accumulator's layout is that of a left operand, what
// one product gives is the next one's operand:
//   x = S k^T,  r = beta (v - e^G x),  n = r T^T,  S <- e^(G_L) S + (e^(G_L - G) n) k
// (all [16][..], tokens or channels as columns).  Of x, r and n each warp has half of the
// tokens; the other warp's half of an operand comes through shared memory, in the order in
// which it lies in registers, while a warp multiplies its own half.  k and T are read from
// shared memory once for both pieces of the left operand.  With its four groups of 16 tokens
// dealt out as {0, 3} and {1, 2}, both warps have as much of the triangle T.
// Of a step's 3800 cycles (backward 5300) the tensor pipes are busy 1400 (2100): the rest is the
// latency of three products, the pieces' rounding and the three meetings of the two warps.
// (2 x 4096 tokens, 16 heads of 128, forward / backward in us: 118 / 165; products shared by 8 or by 16
// warps with barriers between them, bound by reading shared memory, 171 / 231 and 151 / 217;
// one warp to 16 columns, bound by what one warp issues, 164 / 202.)
//
// Backward, what q and do add (E = P^T do and U = (scale e^G q)^T do) does not wait for D: a
// second set of warps forms it beside the ones that carry D.  One more warp loads chunks, two
// stages deep, and one stores the states: the bulk copies' issue alone took a carrying warp
// 500 cycles a chunk.  Every wait is bounded; a warp whose wait ran out asks for nothing and
// arrives nowhere any more (a stage would be asked for before its copies have landed, which its
// barrier does not bear), so that the others' waits run out behind it.
#include <algorithm>

#include "delta_bwd_tc.cuh"

namespace gdn {
namespace {

constexpr int CARRY = 2 * VT / 16;  // warps that carry a state

// In a walk shared memory changes behind barriers that are volatile instructions too, and
// global memory is only written: matrix loads need no more order than among those, and
// products none, so that they can be scheduled into one another.
__device__ __forceinline__ void matrices(uint32_t (&r)[4], const bf16 *row) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0, %1, %2, %3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(ptx::smem_u32(row)));
}
__device__ __forceinline__ void matrices_t(uint32_t (&r)[4], const bf16 *row) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0, %1, %2, %3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(ptx::smem_u32(row)));
}
__device__ __forceinline__ void product(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  asm("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, "
      "{%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
__device__ __forceinline__ void put_matrices(bf16 *row, const uint32_t (&r)[4]) {
  asm volatile("stmatrix.sync.aligned.m8n8.x4.shared.b16 [%0], {%1, %2, %3, %4};" ::"r"(
                   ptx::smem_u32(row)),
               "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]));
}
__device__ __forceinline__ void put_word(uint32_t *to, uint32_t w) {
  asm volatile("st.global.b32 [%0], %1;" ::"l"(__cvta_generic_to_global(to)), "r"(w));
}

// Right operands (two tiles of eight columns) from [n][k] and from [k][n], left ones from
// [k][m].
template <int COLS>
__device__ __forceinline__ void right(uint32_t (&b)[4], const bf16 *s, int n0, int k0) {
  const int l = threadIdx.x & 31;
  matrices(b, s + at<COLS>(n0 + (l & 7) + (l >> 4) * 8, k0 + ((l >> 3) & 1) * 8));
}
template <int COLS>
__device__ __forceinline__ void right_t(uint32_t (&b)[4], const bf16 *s, int n0, int k0) {
  const int l = threadIdx.x & 31;
  matrices_t(b, s + at<COLS>(k0 + (l & 7) + ((l >> 3) & 1) * 8, n0 + (l >> 4) * 8));
}
template <int COLS>
__device__ __forceinline__ void left_t(uint32_t (&a)[4], const bf16 *s, int m0, int k0) {
  const int l = threadIdx.x & 31;
  matrices_t(a, s + at<COLS>(k0 + (l & 7) + (l >> 4) * 8, m0 + ((l >> 3) & 1) * 8));
}
// Where a lane's row of a left operand (16 value columns from row v, columns from c) lies in
// [32][COLS] as 8 x 8 tiles.
template <int COLS>
__device__ __forceinline__ int tile_row(int v, int c) {
  const int l = threadIdx.x & 31;
  return ((v / 8 + ((l >> 3) & 1)) * (COLS / 8) + c / 8 + (l >> 4)) * 64 + (l & 7) * 8;
}
__device__ __forceinline__ void product2(float (*c)[4], const uint32_t (&a)[4], const uint32_t (&b)[4]) {
  product(c[0], a, b[0], b[1]);
  product(c[1], a, b[2], b[3]);
}

// One ring stage's chunk: k, T, values' rows, gates; backward also q and P.
template <int KP, bool BACK>
struct WalkStage {
  static constexpr int K_ = Q * KP * 2, T_ = Block<KP>::SQUARE, V_ = Q * VT * 2, SC_ = Block<KP>::SC;
  static constexpr int Q_AT = K_, T_AT = K_ + (BACK ? K_ : 0), P_AT = T_AT + T_,
                       V_AT = P_AT + (BACK ? T_ : 0), SC_AT = V_AT + V_, BYTES = SC_AT + SC_;
  static constexpr int COPIED = T_ + (BACK ? T_ : 0) + SC_;  // bytes of bulk copies
};

// Shared memory of a walk: two stages; the tiles of S, of r (dn) and of n (dr) by which the
// warps hand on their halves, hi then lo; backward two buffers of E and U for each carrying
// warp.
template <int KP, bool BACK>
struct WalkShared {
  static constexpr int S_AT = 2 * WalkStage<KP, BACK>::BYTES, R_AT = S_AT + Block<KP>::STATE,
                       N_AT = R_AT + Block<KP>::ROWS, HANDS = N_AT + Block<KP>::ROWS;
  static constexpr int HAND = (4 + KP / 16) * 512;
  static constexpr int BYTES = HANDS + (BACK ? 2 * CARRY * HAND : 0);
};

// Element (c, j) of a sequence and head's state tensor.
__device__ __forceinline__ int64_t state_at(const DeltaBwdParams &p, int n, int head, int c, int j) {
  return ((int64_t)n * p.H + head) * p.K * p.V +
         (p.v_first ? (int64_t)j * p.K + c : (int64_t)c * p.V + j);
}

// The first token of sequence n and how many it has.
__device__ __forceinline__ int64_t delta_tokens(const DeltaBwdParams &p, int n, int *len) {
  if (p.cu == nullptr) {
    *len = p.T;
    return (int64_t)n * p.T;
  }
  *len = p.cu[n + 1] - p.cu[n];
  return p.cu[n];
}

// A lane's part of fetching a chunk's rows [64][COLS] (columns from c0 of a tensor
// [.., heads, D]) as an image; zero past `len` rows and past D.
template <int COLS>
__device__ __forceinline__ void fetch_chunk(bf16 *to, const void *tensor, int64_t token, int heads,
                                            int head, int D, int c0, int len) {
  constexpr int EACH = COLS / 8, STEP = 32 / EACH;  // pieces of a row, rows at once
  const int lane = threadIdx.x & 31, col = lane % EACH * 8, first = lane / EACH;
  const int64_t stride = (int64_t)heads * D;
  const bf16 *base = static_cast<const bf16 *>(tensor) + (token * heads + head) * D;
  const bool in = c0 + col < D;
  const bf16 *from = base + (in ? first * stride + c0 + col : 0);
#pragma unroll 4
  for (int r = first; r < Q; r += STEP, from += STEP * stride) {
    const bool ok = in && r < len;
    ptx::cp_async16(to + at<COLS>(r, col), ok ? from : base, ok);
  }
}

// What the roles of a walk share.
template <int KP, bool BACK>
struct Walk {
  using St = WalkStage<KP, BACK>;
  using Sh = WalkShared<KP, BACK>;
  static constexpr int HALF = KP / 2, KS = KP / 32;  // a warp's channels; steps of 16 of them
  unsigned char *shared;
  uint64_t *full, *empty, *ready, *stored, *handed, *taken;
  int vt, v0, head, hk, n, count, len, role, vw, sw, lane, g, t;
  int64_t first, token;
  bool ok;

  __device__ __forceinline__ void wait(uint64_t *bar, int use) {
    // (carry, hand on, load, store)
    const int who = role == 0 ? 0 : BACK && role == 1 ? 1 : 2 + sw;
    ok = ptx::mbar_wait_bounded(bar, (uint32_t)(use & 1), ok ? ptx::role_polls(who) : 1u) && ok;
  }
  __device__ __forceinline__ void arrive(uint64_t *bar) const {
    __syncwarp();
    if (lane == 0 && ok) ptx::mbar_arrive(bar);
  }
  // The two warps of 16 value columns meet.
  __device__ __forceinline__ void meet() const {
    asm volatile("bar.sync %0, 64;" ::"r"(1 + vw) : "memory");
  }
  // the i-th chunk that is taken
  __device__ __forceinline__ int chunk(int i) const { return BACK ? count - 1 - i : i; }
  __device__ __forceinline__ unsigned char *stage(int i) const { return shared + (i & 1) * St::BYTES; }
  template <typename T>
  __device__ __forceinline__ const T *in(int i, int place) const {
    return reinterpret_cast<const T *>(stage(i) + place);
  }
  __device__ __forceinline__ bf16 *tiles(int place) const {
    return reinterpret_cast<bf16 *>(shared + place);
  }
  __device__ __forceinline__ int hand_bar(int i) const { return (i & 1) * CARRY + 2 * vw + sw; }
  __device__ __forceinline__ float4 *hand(int i) const {
    return reinterpret_cast<float4 *>(shared + Sh::HANDS + hand_bar(i) * Sh::HAND) + lane;
  }
  // Warp `s`'s u-th group of 16 tokens.
  __device__ __forceinline__ int group(int s, int u) const { return s ? 1 + u : 3 * u; }

  // The loading warp.
  __device__ __forceinline__ void load(const DeltaBwdParams &p) {
    int i = 0;
    for (; i < count; ++i) {
      if (i >= 2) wait(&empty[i & 1], i / 2 - 1);
      if (!__all_sync(~0u, ok)) break;
      const int c = chunk(i);
      const Block<KP> w(p, first + c, head);
      unsigned char *to = stage(i);
      if (lane == 0) {
        ptx::mbar_arrive_expect_tx(&full[i & 1], St::COPIED);
        ptx::bulk_g2s(to + St::T_AT, w.T(), St::T_ + (BACK ? St::T_ : 0), &full[i & 1]);
        ptx::bulk_g2s(to + St::SC_AT, w.sc(), St::SC_, &full[i & 1]);
      }
      const int64_t at = token + (int64_t)c * Q;
      const int rows = len - c * Q;
      fetch_chunk<KP>(reinterpret_cast<bf16 *>(to), p.k, at, p.Hg, hk, p.K, 0, rows);
      if (BACK)
        fetch_chunk<KP>(reinterpret_cast<bf16 *>(to + St::Q_AT), p.q, at, p.Hg, hk, p.K, 0, rows);
      fetch_chunk<VT>(reinterpret_cast<bf16 *>(to + St::V_AT), BACK ? p.dout : p.v, at, p.H, head,
                      p.V, v0, rows);
      ptx::cp_async_mbar_arrive(&full[i & 1]);
    }
    // the last copies asked for land before the warp ends, whoever else waits for them and
    // whatever ran out
    ptx::cp_async_commit();
    ptx::cp_async_wait<0>();
    for (int k = max(0, i - 2); k < i; ++k)
      ok = ptx::mbar_wait_bounded(&full[k & 1], (uint32_t)(k / 2 & 1), 1u << 22) && ok;
  }

  __device__ __forceinline__ void load_state(const DeltaBwdParams &p, const float *from,
                                             float (*s)[4]) const {
#pragma unroll
    for (int j = 0; j < HALF / 8; ++j)
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const int c = sw * HALF + 8 * j + 2 * t + (e & 1), v = v0 + 16 * vw + g + 8 * (e >> 1);
        s[j][e] = from && c < p.K && v < p.V ? from[state_at(p, n, head, c, v)] : 0.f;
      }
  }

  // x (own tokens) = S k^T of the i-th chunk.  S's pieces go to shared memory, for the other
  // warp and for the storing one.  (All are formed first: the products then follow one another
  // without waiting for a rounding.)
  __device__ __forceinline__ void times_keys(float (*x)[4], const float (*s)[4], const bf16 *k, int i) {
    bf16 *S = tiles(Sh::S_AT);
    uint32_t hi[KS][4], lo[KS][4], b[KS][2][4];
#pragma unroll
    for (int j = 0; j < KS; ++j)
#pragma unroll
      for (int e = 0; e < 4; ++e)
        split(s[2 * j + e / 2][e % 2 * 2], s[2 * j + e / 2][e % 2 * 2 + 1], hi[j][e], lo[j][e]);
    if (i > 0) wait(stored, i - 1);  // the chunk's before has been read
#pragma unroll
    for (int j = 0; j < KS; ++j) {
      put_matrices(S + tile_row<KP>(16 * vw, sw * HALF + 16 * j), hi[j]);
      put_matrices(S + KP * VT + tile_row<KP>(16 * vw, sw * HALF + 16 * j), lo[j]);
    }
    ptx::fence_proxy_async_smem();
    arrive(ready);
#pragma unroll
    for (int half = 0; half < 2; ++half) {
      const int c = (half ? sw ^ 1 : sw) * HALF;
      if (half) {
        meet();
#pragma unroll
        for (int j = 0; j < KS; ++j) {
          matrices(hi[j], S + tile_row<KP>(16 * vw, c + 16 * j));
          matrices(lo[j], S + KP * VT + tile_row<KP>(16 * vw, c + 16 * j));
        }
      }
#pragma unroll
      for (int j = 0; j < KS; ++j)
#pragma unroll
        for (int u = 0; u < 2; ++u) right<KP>(b[j][u], k, 16 * group(sw, u), c + 16 * j);
#pragma unroll
      for (int j = 0; j < KS; ++j) {
#pragma unroll
        for (int u = 0; u < 2; ++u) product2(x + 2 * u, hi[j], b[j][u]);
#pragma unroll
        for (int u = 0; u < 2; ++u) product2(x + 2 * u, lo[j], b[j][u]);
      }
    }
  }

  // The storing warp: a chunk's state as a whole to the workspace.
  template <typename Image>
  __device__ __forceinline__ void store(Image image) {
    for (int i = 0; i < count; ++i) {
      wait(ready, i);
      if (!__all_sync(~0u, ok)) break;
      if (lane == 0) {
        ptx::bulk_s2g(image(i), tiles(Sh::S_AT), Block<KP>::STATE);
        ptx::bulk_commit();
        ptx::bulk_wait_read<0>();
        ptx::mbar_arrive(stored);
      }
      __syncwarp();
    }
    if (lane == 0) ptx::bulk_wait<0>();
  }

  // Hands on own tokens' left operands by `to` (tiles [32][64]); fetches the other warp's.
  __device__ __forceinline__ void give(bf16 *to, const uint32_t (*hi)[4], const uint32_t (*lo)[4]) const {
#pragma unroll
    for (int u = 0; u < 2; ++u) {
      put_matrices(to + tile_row<Q>(16 * vw, 16 * group(sw, u)), hi[u]);
      put_matrices(to + Q * VT + tile_row<Q>(16 * vw, 16 * group(sw, u)), lo[u]);
    }
  }
  __device__ __forceinline__ void take(const bf16 *from, uint32_t (*hi)[4], uint32_t (*lo)[4]) const {
#pragma unroll
    for (int u = 0; u < 2; ++u) {
      matrices(hi[u], from + tile_row<Q>(16 * vw, 16 * group(sw ^ 1, u)));
      matrices(lo[u], from + Q * VT + tile_row<Q>(16 * vw, 16 * group(sw ^ 1, u)));
    }
  }

  // What y (own tokens) += x T^T (backward x T) takes of T, x being warp `s`'s tokens, into the
  // tokens behind (before) them, as T's upper triangle is zero; and the products.
  struct Triangle {
    uint32_t b[2][2][2][4];  // [from][to][piece]
  };
  __device__ __forceinline__ bool within(int from, int to) const { return BACK ? from >= to : from <= to; }
  __device__ __forceinline__ void take_T(Triangle &T, const bf16 *at_, int s) const {
#pragma unroll
    for (int u = 0; u < 2; ++u)
#pragma unroll
      for (int o = 0; o < 2; ++o)
#pragma unroll
        for (int piece = 0; piece < 2; ++piece) {
          const int from = group(s, u), to = group(sw, o);
          if (!within(from, to)) continue;
          if (BACK)
            right_t<64>(T.b[u][o][piece], at_ + piece * Q * Q, 16 * to, 16 * from);
          else
            right<64>(T.b[u][o][piece], at_ + piece * Q * Q, 16 * to, 16 * from);
        }
  }
  __device__ __forceinline__ void times_T(float (*y)[4], const uint32_t (*hi)[4],
                                          const uint32_t (*lo)[4], const Triangle &T, int s) const {
#pragma unroll
    for (int u = 0; u < 2; ++u)
#pragma unroll
      for (int piece = 0; piece < 3; ++piece)
#pragma unroll
        for (int o = 0; o < 2; ++o) {
          if (!within(group(s, u), group(sw, o))) continue;
          product2(y + 2 * o, piece == 1 ? lo[u] : hi[u], T.b[u][o][piece == 2]);
        }
  }

  // s (own channels) += a rows: a [16][warp `from`'s tokens] as pieces, rows [64][KP].
  __device__ __forceinline__ void add_outer(float (*s)[4], const uint32_t (*hi)[4],
                                            const uint32_t (*lo)[4], const bf16 *rows, int from) const {
#pragma unroll
    for (int u = 0; u < 2; ++u) {
      uint32_t b[KS][4];
#pragma unroll
      for (int j = 0; j < KS; ++j) right_t<KP>(b[j], rows, sw * HALF + 16 * j, 16 * group(from, u));
#pragma unroll
      for (int j = 0; j < KS; ++j) product2(s + 2 * j, hi[u], b[j]);
#pragma unroll
      for (int j = 0; j < KS; ++j) product2(s + 2 * j, lo[u], b[j]);
    }
  }

  // Own tokens' values to the workspace's image [32][64], both pieces.
  __device__ __forceinline__ void keep_tiles(unsigned char *image, const float (*y)[4]) const {
    uint32_t *word = reinterpret_cast<uint32_t *>(image) + 2 * vw * 8 * 32 + lane;
#pragma unroll
    for (int j = 0; j < 4; ++j)
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        uint32_t hi, lo;
        split(y[j][2 * e], y[j][2 * e + 1], hi, lo);
        const int tile = e * 8 + 2 * group(sw, j / 2) + j % 2;
        put_word(word + tile * 32, hi);
        put_word(word + tile * 32 + Q * VT / 2, lo);
      }
  }

  // Pairs of a chunk's gates at own tokens: tile j's columns.
  __device__ __forceinline__ float2 pair(const float *of, int j) const {
    return *reinterpret_cast<const float2 *>(of + 16 * group(sw, j / 2) + 8 * (j % 2) + 2 * t);
  }
};

// The pieces of own tokens' accumulators, each column by its token's factor, as left operands.
template <typename F>
__device__ __forceinline__ void to_operand(const float (*y)[4], uint32_t (*hi)[4], uint32_t (*lo)[4],
                                           F factor) {
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    const float2 f = factor(j);
#pragma unroll
    for (int e = 0; e < 2; ++e)
      split(f.x * y[j][2 * e], f.y * y[j][2 * e + 1], hi[j / 2][j % 2 * 2 + e],
            lo[j / 2][j % 2 * 2 + e]);
  }
}

// The roles: warps 0 .. CARRY - 1 carry states; backward CARRY more hand them E and U; the last
// two load and store.  Returns false where there is nothing to do.
template <int KP, bool BACK>
__device__ __forceinline__ bool begin_walk(const DeltaBwdParams &p, Walk<KP, BACK> &w,
                                           unsigned char *shared, uint64_t *bars) {
  const int warp = threadIdx.x >> 5;
  w.shared = shared;
  w.full = bars;
  w.empty = bars + 2;
  w.ready = bars + 4;
  w.stored = bars + 5;
  w.handed = bars + 6;
  w.taken = bars + 6 + 2 * CARRY;
  w.vt = blockIdx.x;
  w.v0 = w.vt * VT;
  w.head = blockIdx.y;
  w.hk = w.head / (p.H / p.Hg);
  w.role = warp / CARRY;
  w.vw = warp % CARRY / 2;
  w.sw = warp % 2;
  w.lane = threadIdx.x & 31;
  w.g = w.lane >> 2;
  w.t = w.lane & 3;
  w.ok = true;
  ptx::griddep_wait();
  if (!delta_good(p)) return false;
  w.n = delta_turn(p, blockIdx.z);
  w.count = delta_chunks(p, w.n, &w.first);
  if (!bounds_ok(w.v0 < p.V && w.head < p.H && w.n < p.N && w.first + w.count <= p.chunks, p.err))
    return false;
  w.token = delta_tokens(p, w.n, &w.len);
  if (threadIdx.x == 0) {
    for (int s = 0; s < 2; ++s) {
      ptx::mbar_init(&w.full[s], 33);
      ptx::mbar_init(&w.empty[s], BACK ? 2 * CARRY : CARRY);
    }
    ptx::mbar_init(w.ready, CARRY);
    ptx::mbar_init(w.stored, 1);
    if (BACK)
      for (int s = 0; s < 2 * CARRY; ++s) {
        ptx::mbar_init(&w.handed[s], 1);
        ptx::mbar_init(&w.taken[s], 1);
      }
    ptx::fence_mbar_init();
  }
  __syncthreads();
  return true;
}

// grid: value tiles, heads, sequences.  The states, forward.
template <int KP>
__global__ void __launch_bounds__(32 * (CARRY + 2), 2) tc_states_kernel(DeltaBwdParams p) {
  using W = Walk<KP, false>;
  using St = WalkStage<KP, false>;
  extern __shared__ __align__(128) unsigned char shared[];
  __shared__ uint64_t bars[6];
  W w;
  if (!begin_walk(p, w, shared, bars)) return;
  if (w.role == 1 && w.vw == 0) {
    if (w.sw == 0)
      w.load(p);
    else
      w.store([&](int i) { return Block<KP>(p, w.first + i, w.head).h(w.vt); });
  } else {
    bf16 *R = w.tiles(W::Sh::R_AT), *N = w.tiles(W::Sh::N_AT);
    float s[W::HALF / 8][4];
    w.load_state(p, p.h0, s);
    for (int c = 0; c < w.count; ++c) {
      const Block<KP> block(p, w.first + c, w.head);
      w.wait(&w.full[c & 1], c / 2);
      const bf16 *k = w.template in<bf16>(c, 0), *T = w.template in<bf16>(c, St::T_AT);
      const bf16 *v = w.template in<bf16>(c, St::V_AT);
      const float *sc = w.template in<float>(c, St::SC_AT);
      const float *beta = sc + Q, *eG = sc + 2 * Q, *eR = sc + 3 * Q;
      float x[4][4] = {}, y[4][4] = {};
      uint32_t hi[2][4], lo[2][4], b[4];
      typename W::Triangle own, other;
      w.times_keys(x, s, k, c);
      w.take_T(own, T, w.sw);
      w.take_T(other, T, w.sw ^ 1);
#pragma unroll
      for (int u = 0; u < 2; ++u) {  // the values as the accumulators have them
        left_t<32>(b, v, 16 * w.vw, 16 * w.group(w.sw, u));
#pragma unroll
        for (int j = 0; j < 2; ++j) {
          const float2 f = w.pair(beta, 2 * u + j), e = w.pair(eG, 2 * u + j);
#pragma unroll
          for (int r = 0; r < 2; ++r) {
            const float *a = x[2 * u + j] + 2 * r;
            const float2 val = __bfloat1622float2(*reinterpret_cast<const __nv_bfloat162 *>(&b[2 * j + r]));
            split(f.x * fmaf(-e.x, a[0], val.x), f.y * fmaf(-e.y, a[1], val.y), hi[u][2 * j + r],
                  lo[u][2 * j + r]);
          }
        }
      }
      w.give(R, hi, lo);
      w.times_T(y, hi, lo, own, w.sw);
      w.meet();
      w.take(R, hi, lo);
      w.times_T(y, hi, lo, other, w.sw ^ 1);
      if (c + 1 < w.count) {
        to_operand(y, hi, lo, [&](int j) { return w.pair(eR, j); });
        w.give(N, hi, lo);
        const float eL = eG[Q - 1];
#pragma unroll
        for (int j = 0; j < W::HALF / 8; ++j)
#pragma unroll
          for (int e = 0; e < 4; ++e) s[j][e] *= eL;
        w.add_outer(s, hi, lo, k, w.sw);
        w.keep_tiles(block.n(w.vt), y);
        w.meet();
        w.take(N, hi, lo);
        w.add_outer(s, hi, lo, k, w.sw ^ 1);
      } else {
        w.keep_tiles(block.n(w.vt), y);
      }
      w.arrive(&w.empty[c & 1]);
    }
  }
  if (!w.ok && w.lane == 0) record_error(p.err, GDN_ERR_TIMEOUT);
}

// grid: as tc_states_kernel, from the last chunk to the first: with E and U
//   x = D k^T,  dn = E + e^(G_L - G) x,  dr = dn T,  D <- e^(G_L) D + U - (beta e^G dr) k.
// dv = beta dr leaves from here too.
template <int KP>
__global__ void __launch_bounds__(32 * (2 * CARRY + 2), 1) tc_grads_kernel(DeltaBwdParams p) {
  using W = Walk<KP, true>;
  using St = WalkStage<KP, true>;
  extern __shared__ __align__(128) unsigned char shared[];
  __shared__ uint64_t bars[6 + 4 * CARRY];
  W w;
  if (!begin_walk(p, w, shared, bars)) return;
  if (w.role == 2) {
    if (w.sw == 0)
      w.load(p);
    else
      w.store([&](int i) { return Block<KP>(p, w.first + w.chunk(i), w.head).D(w.vt); });
  } else if (w.role == 1) {  // E of own tokens and U of own channels
    for (int i = 0; i < w.count; ++i) {
      w.wait(&w.full[i & 1], i / 2);
      const bf16 *q = w.template in<bf16>(i, St::Q_AT), *P = w.template in<bf16>(i, St::P_AT);
      const bf16 *go = w.template in<bf16>(i, St::V_AT);
      const float *eG = w.template in<float>(i, St::SC_AT) + 2 * Q + 2 * w.t;
      float E[4][4] = {}, U[W::HALF / 8][4] = {};
#pragma unroll
      for (int kk = 0; kk < 4; ++kk) {
        uint32_t a[4], b[4], hi[4], lo[4], rows[W::KS][4];
        left_t<32>(a, go, 16 * w.vw, 16 * kk);
#pragma unroll
        for (int j = 0; j < W::KS; ++j) right_t<KP>(rows[j], q, w.sw * W::HALF + 16 * j, 16 * kk);
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const float2 f = *reinterpret_cast<const float2 *>(eG + 16 * kk + 8 * (e / 2));
          const float2 d = __bfloat1622float2(*reinterpret_cast<const __nv_bfloat162 *>(&a[e]));
          split(p.scale * f.x * d.x, p.scale * f.y * d.y, hi[e], lo[e]);
        }
#pragma unroll
        for (int j = 0; j < W::KS; ++j) product2(U + 2 * j, hi, rows[j]);
#pragma unroll
        for (int piece = 0; piece < 2; ++piece)
#pragma unroll
          for (int o = 0; o < 2; ++o) {
            const int to = w.group(w.sw, o);
            if (kk < to) continue;
            right_t<64>(b, P + piece * Q * Q, 16 * to, 16 * kk);
            product2(E + 2 * o, a, b);
          }
#pragma unroll
        for (int j = 0; j < W::KS; ++j) product2(U + 2 * j, lo, rows[j]);
      }
      if (i >= 2) w.wait(&w.taken[w.hand_bar(i)], i / 2 - 1);
      float4 *to = w.hand(i);
#pragma unroll
      for (int j = 0; j < 4; ++j) to[j * 32] = make_float4(E[j][0], E[j][1], E[j][2], E[j][3]);
#pragma unroll
      for (int j = 0; j < W::HALF / 8; ++j)
        to[(4 + j) * 32] = make_float4(U[j][0], U[j][1], U[j][2], U[j][3]);
      w.arrive(&w.handed[w.hand_bar(i)]);
      w.arrive(&w.empty[i & 1]);
    }
  } else {
    bf16 *R = w.tiles(W::Sh::R_AT), *N = w.tiles(W::Sh::N_AT);
    float s[W::HALF / 8][4];
    w.load_state(p, p.dht, s);
    for (int i = 0; i < w.count; ++i) {
      const int c = w.chunk(i);
      const Block<KP> block(p, w.first + c, w.head);
      w.wait(&w.full[i & 1], i / 2);
      const bf16 *k = w.template in<bf16>(i, 0), *T = w.template in<bf16>(i, St::T_AT);
      const float *sc = w.template in<float>(i, St::SC_AT);
      const float *beta = sc + Q, *eG = sc + 2 * Q, *eR = sc + 3 * Q;
      float x[4][4] = {}, y[4][4] = {};
      uint32_t hi[2][4], lo[2][4];
      typename W::Triangle own, other;
      w.times_keys(x, s, k, i);
      w.take_T(own, T, w.sw);
      w.take_T(other, T, w.sw ^ 1);
      w.wait(&w.handed[w.hand_bar(i)], i / 2);
      const float4 *from = w.hand(i);
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const float2 f = w.pair(eR, j);
        const float4 E = from[j * 32];
        x[j][0] = fmaf(f.x, x[j][0], E.x);
        x[j][1] = fmaf(f.y, x[j][1], E.y);
        x[j][2] = fmaf(f.x, x[j][2], E.z);
        x[j][3] = fmaf(f.y, x[j][3], E.w);
      }
      to_operand(x, hi, lo, [](int) { return make_float2(1.f, 1.f); });
      w.give(R, hi, lo);
      w.times_T(y, hi, lo, own, w.sw);
      const float eL = eG[Q - 1];
#pragma unroll
      for (int j = 0; j < W::HALF / 8; ++j) {
        const float4 U = from[(4 + j) * 32];
        s[j][0] = fmaf(eL, s[j][0], U.x);
        s[j][1] = fmaf(eL, s[j][1], U.y);
        s[j][2] = fmaf(eL, s[j][2], U.z);
        s[j][3] = fmaf(eL, s[j][3], U.w);
      }
      w.arrive(&w.taken[w.hand_bar(i)]);
      w.meet();
      w.take(R, hi, lo);
      w.times_T(y, hi, lo, other, w.sw ^ 1);
      to_operand(y, hi, lo, [&](int j) {
        const float2 f = w.pair(beta, j), e = w.pair(eG, j);
        return make_float2(-f.x * e.x, -f.y * e.y);
      });
      w.give(N, hi, lo);
      w.add_outer(s, hi, lo, k, w.sw);
      w.keep_tiles(block.dr(w.vt), y);
      w.meet();
      w.take(N, hi, lo);
      w.add_outer(s, hi, lo, k, w.sw ^ 1);
      // dv [token][v]: pairs of tokens to pairs of values
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const float2 f = w.pair(beta, j);
        const int row = c * Q + 16 * w.group(w.sw, j / 2) + 8 * (j % 2) + w.g;
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          const __nv_bfloat162 d = __floats2bfloat162_rn(f.x * y[j][2 * e], f.y * y[j][2 * e + 1]);
          const uint32_t word = ptx::transpose_8x8(*reinterpret_cast<const uint32_t *>(&d));
          const int col = w.v0 + 16 * w.vw + 8 * e + 2 * w.t;
          if (row < w.len && col < p.V)
            put_word(reinterpret_cast<uint32_t *>(static_cast<bf16 *>(p.dv) +
                                                  ((w.token + row) * p.H + w.head) * p.V + col),
                     word);
        }
      }
      w.arrive(&w.empty[i & 1]);
    }
    if (p.dh0 != nullptr)
#pragma unroll
      for (int j = 0; j < W::HALF / 8; ++j)
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const int c = w.sw * W::HALF + 8 * j + 2 * w.t + (e & 1);
          const int v = w.v0 + 16 * w.vw + w.g + 8 * (e >> 1);
          if (c < p.K && v < p.V) p.dh0[state_at(p, w.n, w.head, c, v)] = s[j][e];
        }
  }
  if (!w.ok && w.lane == 0) record_error(p.err, GDN_ERR_TIMEOUT);
}

template <int KP>
cudaError_t launch(const DeltaBwdParams &p, cudaStream_t stream) {
  constexpr int STATES = WalkShared<KP, false>::BYTES, GRADS = WalkShared<KP, true>::BYTES;
  cudaError_t e = cudaFuncSetAttribute(tc_states_kernel<KP>,
                                       cudaFuncAttributeMaxDynamicSharedMemorySize, STATES);
  if (e == cudaSuccess)
    e = cudaFuncSetAttribute(tc_grads_kernel<KP>, cudaFuncAttributeMaxDynamicSharedMemorySize, GRADS);
  if (e != cudaSuccess) return e;
  const dim3 grid((p.V + VT - 1) / VT, p.H, p.N);
  e = launch_behind(tc_states_kernel<KP>, grid, 32 * (CARRY + 2), STATES, stream, p);
  if (e != cudaSuccess) return e;
  return launch_behind(tc_grads_kernel<KP>, grid, 32 * (2 * CARRY + 2), GRADS, stream, p);
}

}  // namespace

cudaError_t launch_delta_walks(const DeltaBwdParams &p, cudaStream_t stream) {
  return p.K <= 64 ? launch<64>(p, stream) : launch<128>(p, stream);
}

}  // namespace gdn
