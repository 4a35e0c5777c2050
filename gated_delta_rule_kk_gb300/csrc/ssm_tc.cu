// The state space scan over prompts on the 5th-generation tensor cores, bf16
// tokens, K <= 128 and V in 64-column tiles.
//
// A chunk of Q = 128 tokens of one head.  With G_i the running sum of the
// log-decays a s_t inside the chunk and h the state at its start,
//   Y = diag(e^(G_i)) (C h^T) + M X,   M_ij = (C B^T)_ij e^(G_i - G_j) s_j, j <= i
//   h^T <- e^(G_Q) h^T + B^T W,        W_j = s_j e^(G_Q - G_j) x_j
// that is four products with 128 rows: S = C B^T (N = 128), C h^T (N = 64, h as two
// bf16 pieces along the keys), M X (N = 64, M as two pieces) and B^T W (N = 128 +
// 64: W as three pieces, so that the float32 state gains no rounding from the
// operands).  x, B and C are bf16 themselves and enter exactly.  One piece each of
// h and M left y up to 3e-2 of its RMS off; two leave 16 bits: 2^-16 of the terms'
// magnitudes, 2.4e-6 of y in norm, of a float32 y too (of those rounded to bf16 one in
// 800 is then the neighbour of the exact one's).  A third piece would take 64 more
// columns of TMEM a chunk and another 16 KB, and both are used up.
//
// One CTA per (64-column V tile, head, segment of a sequence) walks the
// segment's chunks; h stays in registers in float32.  S, M and W do not depend
// on h, so only the update of h is sequential.  32 warps, one role each:
//   0-7    M      thread (row i, 16 of every 32 columns): S from TMEM, times
//                 e^(G_i - G_j) s_j, plus D on the diagonal, back over S as the two
//                 bf16 A operands of M X
//   8-15   output thread (row i, 32 columns): y times the gate (whose z comes
//                 straight to registers) into a tile that leaves by TMA
//   16-23  state  thread (key k, 32 columns): h, its bf16 pieces for C h^T; and,
//                 (row i, 32 columns) of C h^T times e^(G_i) in place, where M X
//                 adds to it
//   24-27  W      thread j: row j of the three pieces
//   28     loads  TMA: two x, two B tiles and one C tile (x, C and z of later
//                 chunks asked into L2 before their tiles are free)
//   29     MMA    per chunk B^T W, S of the next chunk, M X, then C h^T of the next:
//                 an order in which each product's operands are formed while the
//                 others run
//   30     scalars  step sizes, log-decays and their sums
//   31     store  TMA: y
// What bounds it (2 x 4096 tokens, 64 heads of 64 x 128, B and C shared by all: 98
// to 101 us, where the bytes alone would take 31 at the copy rate and CUDA cores
// took 1620): 128 CTAs with some 6000 cycles a chunk, in which every role is busy
// for 3000 to 5000, waiting the rest for one another.  The warps' 14900
// instructions a chunk take 65% of an SM's issue slots, the products 40% of the
// tensor pipe, HBM 23% of its rate: fewer instructions a chunk would be the next
// step.  Two y in TMEM (111 us with one, which M X of a chunk shared with the output
// of the one before) and z past shared memory (its tile waited for y's store) keep
// the output out of that chain.
// The decays: every 32-token block b keeps f_j = s_j e^(block end - G_j) and the
// sums inside the block, so that e^(G_i - G_j) s_j is a product of f_j and one
// factor per row and block, all exponents sums of the terms between j and i.  Only on
// the diagonal does the row's factor take what f_j has past i off again: a difference
// of sums of at most 80, of which some 1e-5 is lost at worst.  Where a block decays by
// more, so that the factor could overflow, its elements take an exponential each, of
// sums in fixed point: differences of float32 sums of 1e5 (one token that resets the
// state) had y off by a percent.  (80 or 60 as the limit, us: 98 / 105, 283 / 317 for
// eight packed prompts: the heads of the strongest decays set the pace.)
//
// Every wait is bounded: a role whose wait runs out issues nothing more and ends
// after its step, GDN_ERR_TIMEOUT is recorded, the copies and products that are on
// their way are waited for and the block returns.
#include "ptx.cuh"
#include "rows.cuh"
#include "ssm_items.cuh"
#include "tensor_map.h"

namespace gdn {
namespace {

constexpr int ST_Q = 128, ST_VT = 64;
// first warp of each role after M's
constexpr int ST_W_OUT = 8, ST_W_STATE = 16, ST_W_W = 24, ST_W_LOAD = 28, ST_W_MMA = 29,
              ST_W_SCALARS = 30, ST_THREADS = 32 * 32;
// Registers of a thread of each role.  The block starts with 64 a thread, and
// 64 + 64 + 64 + 64 + 80 + 80 + 48 + 48, the warpgroups' shares, is what 8
// warpgroups have at 64 (16 bytes of spills are left in all).
constexpr int ST_R_STATE = 80, ST_R_W = 48, ST_R_REST = 48;
static_assert(4 * 64 + 2 * ST_R_STATE + ST_R_W + ST_R_REST <= 8 * 64, "registers");
constexpr uint32_t ST_TILE = 16384;  // 128 rows of 128 bytes, 128-byte swizzle
// TMEM columns: two of S, then M over it (16 columns of S hold 8 of M's high and
// 8 of its low pieces, bf16 pairs); two of y, which starts as C h^T; B^T W, the
// first piece and the sum of the others
constexpr uint32_t ST_S = 0, ST_Y = 256, ST_DH = 384;

// Per-chunk scalars, two buffers.
struct StScalars {
  float f[ST_Q];    // s_j e^(sum of the block's log-decays after j)
  float pin[ST_Q];  // log-decays of the block up to and with i
  float tb[4];      // the blocks' sums
  float sfx[4];     // e^(sums of the later blocks)
  float total;      // the chunk's sum
  float pad[7];
};

// A wait sees a phase by its parity, so a barrier may complete a phase only after
// every role has seen the one before: one barrier for each of two buffers, or one
// whose next phase needs something of all its waiters first.
struct StBars {
  uint64_t x_full[2], x_free[2], b_full[2], b_free[2], sc_full[2], sc_free[2], s_full[2],
      ready[2], y_full[2], y_read[2];
  uint64_t y_sent, off_full, w_full, dh_full, dh_free, h_full, staged,
      drained;
};

// The first token of the segment, counted from its start, whose x is not finite in
// each of the tile's columns, and the least of them.  The zeros of M past the
// diagonal would carry such an x to the tokens before it (0 x Inf = NaN), so it
// enters M X as zero and the output writes NaN from its token on.
struct StBad {
  int first[ST_VT], any;
};
constexpr int ST_NEVER = 0x7fffffff;

template <int KH>  // 64-key halves of a B or C tile
struct StLayout {
  static constexpr uint32_t X = 0, Y = 2 * ST_TILE, B = 3 * ST_TILE, C = B + 2 * KH * ST_TILE;
  static constexpr uint32_t W = C + KH * ST_TILE, H = W + 3 * ST_TILE, SC = H + 2 * ST_TILE;
  static constexpr uint32_t BARS = SC + 2 * sizeof(StScalars);
  static constexpr uint32_t BAD = BARS + sizeof(StBars) + 16;
  static constexpr uint32_t BYTES = BAD + sizeof(StBad);
};
static_assert(StLayout<2>::BYTES <= 232448, "shared memory of one CTA");

// Byte of 16-byte piece c of row r in a 128-byte swizzled tile.
__device__ __forceinline__ uint32_t swz(int r, int c) { return r * 128 + ((c ^ (r & 7)) << 4); }

__device__ __forceinline__ void tma_load_4d(void *dst, const void *tmap, int c0, int c1, int c2,
                                            int c3, uint64_t *bar) {
  asm volatile(
      "cp.async.bulk.tensor.4d.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
      " [%0], [%1, {%2, %3, %4, %5}], [%6];" ::"r"(ptx::smem_u32(dst)),
      "l"(tmap), "r"(c0), "r"(c1), "r"(c2), "r"(c3), "r"(ptx::smem_u32(bar))
      : "memory");
}
// Asks a box into L2.
__device__ __forceinline__ void tma_prefetch_4d(const void *tmap, int c0, int c1, int c2, int c3) {
  asm volatile("cp.async.bulk.prefetch.tensor.4d.L2.global.tile [%0, {%1, %2, %3, %4}];" ::"l"(tmap),
               "r"(c0), "r"(c1), "r"(c2), "r"(c3)
               : "memory");
}
__device__ __forceinline__ void tma_store_4d(const void *tmap, int c0, int c1, int c2, int c3,
                                             const void *src) {
  asm volatile(
      "cp.async.bulk.tensor.4d.global.shared::cta.tile.bulk_group [%0, {%1, %2, %3, %4}], [%5];" ::
          "l"(tmap),
      "r"(c0), "r"(c1), "r"(c2), "r"(c3), "r"(ptx::smem_u32(src))
      : "memory");
}

// The tensor-core instructions below are issued by the lane with `one` set and
// are reached by the whole warp: without a branch around them their operands
// stay in uniform registers, and an instruction costs less to issue.
__device__ __forceinline__ uint32_t elect_one() {
  uint32_t one;
  asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.u32 %0, 1, 0, p;\n\t}"
               : "=r"(one));
  return one;
}
// D[tmem] (+)= A * B[smem], bf16 operands, fp32 accumulate; A in shared memory
// or in tensor memory.  Operands in shared memory by the low word of their
// descriptor (all share the high one): one 32-bit addition leads to the next.
constexpr uint32_t ST_DESC_HIGH = (1024 >> 4) | 1u << 14 | 2u << 29;
__device__ __forceinline__ void mma_ss(uint32_t one, uint32_t d_tmem, uint32_t a, uint32_t b,
                                       uint32_t idesc, uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p, q;\n\t.reg .b64 da, db;\n\tsetp.ne.b32 p, %4, 0;\n\t"
      "setp.ne.b32 q, %5, 0;\n\tmov.b64 da, {%1, %6};\n\tmov.b64 db, {%2, %6};\n\t"
      "@q tcgen05.mma.cta_group::1.kind::f16 [%0], da, db, %3, p;\n\t}" ::"r"(d_tmem),
      "r"(a), "r"(b), "r"(idesc), "r"(accumulate), "r"(one), "r"(ST_DESC_HIGH)
      : "memory");
}
__device__ __forceinline__ void mma_ts(uint32_t one, uint32_t d_tmem, uint32_t a_tmem, uint32_t b,
                                       uint32_t idesc, uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p, q;\n\t.reg .b64 db;\n\tsetp.ne.b32 p, %4, 0;\n\t"
      "setp.ne.b32 q, %5, 0;\n\tmov.b64 db, {%2, %6};\n\t"
      "@q tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], db, %3, p;\n\t}" ::"r"(d_tmem),
      "r"(a_tmem), "r"(b), "r"(idesc), "r"(accumulate), "r"(one), "r"(ST_DESC_HIGH)
      : "memory");
}
__device__ __forceinline__ void commit(uint32_t one, uint64_t *bar) {
  asm volatile(
      "{\n\t.reg .pred q;\n\tsetp.ne.b32 q, %1, 0;\n\t"
      "@q tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];\n\t}" ::"r"(
          ptx::smem_u32(bar)),
      "r"(one)
      : "memory");
}

// 16 consecutive 32-bit columns of this thread's TMEM lane.
__device__ __forceinline__ void tmem_st16(uint32_t taddr, const uint32_t *r) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x16.b32 [%16], {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,"
      "%13,%14,%15};" ::"r"(r[0]),
      "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]),
      "r"(r[9]), "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15]), "r"(taddr)
      : "memory");
}
// 8 of them.
__device__ __forceinline__ void tmem_st8(uint32_t taddr, const uint32_t *r) {
  asm volatile("tcgen05.st.sync.aligned.32x32b.x8.b32 [%8], {%0,%1,%2,%3,%4,%5,%6,%7};" ::"r"(r[0]),
               "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]),
               "r"(taddr)
               : "memory");
}
__device__ __forceinline__ void tmem_wait_st() {
  asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory");
}
__device__ __forceinline__ void tmem_wait_ld() {
  asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory");
}
// Keeps the compiler from using the registers before this point.
template <int N>
__device__ __forceinline__ void pin_regs(uint32_t *r) {
#pragma unroll
  for (int i = 0; i < N; ++i) asm volatile("" : "+r"(r[i]));
}
// Loads whose registers are valid after tmem_wait_ld (then pin_regs).
__device__ __forceinline__ void tmem_ld16_async(uint32_t taddr, uint32_t *r) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,"
      "%14,%15}, [%16];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]),
        "=r"(r[7]), "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]),
        "=r"(r[14]), "=r"(r[15])
      : "r"(taddr)
      : "memory");
}
__device__ __forceinline__ void tmem_ld8_async(uint32_t taddr, uint32_t *r) {
  asm volatile("tcgen05.ld.sync.aligned.32x32b.x8.b32 {%0,%1,%2,%3,%4,%5,%6,%7}, [%8];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]),
                 "=r"(r[6]), "=r"(r[7])
               : "r"(taddr)
               : "memory");
}

// mbar_wait_bounded as one short loop: this kernel's roles meet at some forty
// barriers, and its code has to stay in the instruction cache.
__device__ __forceinline__ bool wait_bounded(uint64_t *bar, uint32_t parity, uint32_t tries) {
  uint32_t left;
  asm volatile(
      "{\n\t.reg .pred p, q;\n\tmov.u32 %0, %3;\n\t"
      "WAIT:\n\tmbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2;\n\t@p bra DONE;\n\t"
      "sub.u32 %0, %0, 1;\n\tsetp.ne.u32 q, %0, 0;\n\t@q bra WAIT;\n\tDONE:\n\t}"
      : "=&r"(left)
      : "r"(ptx::smem_u32(bar)), "r"(parity), "r"(tries)
      : "memory");
  return left != 0;
}

// This warpgroup's registers a thread (all four warps call it).
template <int N>
__device__ __forceinline__ void regs_up() {
  asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(N));
}
template <int N>
__device__ __forceinline__ void regs_down() {
  asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(N));
}

__device__ __forceinline__ uint32_t pack2(float a, float b) {
  const __nv_bfloat162 h = __floats2bfloat162_rn(a, b);
  return *reinterpret_cast<const uint32_t *>(&h);
}
__device__ __forceinline__ float low(uint32_t w) { return __uint_as_float(w << 16); }
__device__ __forceinline__ float high(uint32_t w) { return __uint_as_float(w & 0xffff0000u); }

// Low word of the descriptor of a 128-byte swizzled operand, `lbo` bytes between
// its halves, and the word `bytes` further on.
__device__ __forceinline__ uint32_t sw128(const void *smem, uint32_t lbo) {
  return (ptx::smem_u32(smem) >> 4) | lbo << 12;
}
__device__ __forceinline__ uint32_t ahead(uint32_t desc, uint32_t bytes) { return desc + (bytes >> 4); }

// STATES: the first of two passes, which keeps only every segment's last state.
template <int KH, bool STATES>
__global__ void __launch_bounds__(ST_THREADS, 1)
ssm_tc_kernel(const __grid_constant__ CUtensorMap tm_x, const __grid_constant__ CUtensorMap tm_b,
              const __grid_constant__ CUtensorMap tm_c, const __grid_constant__ CUtensorMap tm_z,
              const __grid_constant__ CUtensorMap tm_y, SsmParams p) {
  extern __shared__ __align__(1024) unsigned char sm[];
  using L = StLayout<KH>;
  StScalars *sc = reinterpret_cast<StScalars *>(sm + L::SC);
  StBars &bar = *reinterpret_cast<StBars *>(sm + L::BARS);
  uint32_t *tmem_slot = reinterpret_cast<uint32_t *>(sm + L::BARS + sizeof(StBars));
  StBad &bad = *reinterpret_cast<StBad *>(sm + L::BAD);
  // (a warp's index the compiler knows to be the same in all its lanes, so that
  // each role's addresses and descriptors live in uniform registers)
  const int tid = threadIdx.x, warp = __shfl_sync(~0u, tid >> 5, 0), lane = tid & 31;
  const int vtiles = (p.V + ST_VT - 1) / ST_VT;
  const int h = blockIdx.x / vtiles, v0 = (blockIdx.x % vtiles) * ST_VT, g = h / (p.H / p.Hg);
  if (!offsets_ok(p.cu, p.N, p.T, p.err)) return;
  const int item = blockIdx.y;
  const SsmItem q = ssm_item(p, item);
  if (q.n < 0 || (STATES && q.last)) return;
  if (!bounds_ok(q.n < p.N && q.lo >= 0 && q.lo <= q.hi && q.hi <= p.T && h < p.H &&
                     (ptx::smem_u32(sm) & 1023u) == 0,
                 p.err))
    return;
  const int nch = (q.hi - q.lo + ST_Q - 1) / ST_Q;
  const int K = p.K, V = p.V, width = min(ST_VT, V - v0);

  if (tid == 0) {
    for (int s = 0; s < 2; ++s) {
      ptx::mbar_init(&bar.x_full[s], 1);
      ptx::mbar_init(&bar.x_free[s], 1);
      ptx::mbar_init(&bar.b_full[s], STATES ? 1 : 2);  // B, and C
      ptx::mbar_init(&bar.b_free[s], 1);
      ptx::mbar_init(&bar.sc_full[s], 1);
      ptx::mbar_init(&bar.s_full[s], 1);
      ptx::mbar_init(&bar.ready[s], 16);  // M, and C h^T scaled
      ptx::mbar_init(&bar.y_full[s], 1);
      ptx::mbar_init(&bar.y_read[s], 8);
      ptx::mbar_init(&bar.sc_free[s], STATES ? 12 : 20);  // the warps that read them
    }
    ptx::mbar_init(&bar.y_sent, 1);
    ptx::mbar_init(&bar.off_full, 1);
    ptx::mbar_init(&bar.w_full, 4);
    ptx::mbar_init(&bar.dh_full, 1);
    ptx::mbar_init(&bar.dh_free, 8);
    ptx::mbar_init(&bar.h_full, 8);
    ptx::mbar_init(&bar.staged, 8);
    ptx::mbar_init(&bar.drained, 1);
    ptx::fence_mbar_init();
  }
  if (!STATES && tid <= ST_VT) (tid < ST_VT ? bad.first[tid] : bad.any) = ST_NEVER;
  if (warp == 0) ptx::tmem_alloc<512>(tmem_slot);
  ptx::tc_fence_before();
  __syncthreads();
  ptx::tc_fence_after();
  const uint32_t tmem = __shfl_sync(~0u, *tmem_slot, 0);
  const uint32_t lanes = (uint32_t)((warp & 3) * 32) << 16;  // this warp's TMEM lanes
  bool ok = true;
  auto wait = [&](uint64_t *b, int phase) {
    ok = wait_bounded(b, (uint32_t)(phase & 1), ok ? 1u << 22 : 1u) && ok;
  };
  // a wait of its own: what it waits for comes whatever went wrong elsewhere
  auto drain = [&](uint64_t *b, int phase) {
    ok = wait_bounded(b, (uint32_t)(phase & 1), 1u << 22) && ok;
  };
  auto arrive = [&](uint64_t *b) {
    __syncwarp();
    if (lane == 0) ptx::mbar_arrive(b);
  };
  auto going = [&] { return __all_sync(~0u, ok) != 0; };
  auto tokens_of = [&](int it) { return min(ST_Q, q.hi - q.lo - it * ST_Q); };

  if (warp < ST_W_OUT) {
    // ---------------- M
    const int w4 = warp & 3, i = 32 * w4 + lane, c = 16 * (warp >> 2);
    const float skip = p.D ? p.D[h] : 0.f;
#pragma unroll 1
    for (int it = 0; it < (STATES ? 0 : nch) && going(); ++it) {
      const StScalars &s = sc[it & 1];
      const int n = tokens_of(it);
      wait(&bar.sc_full[it & 1], it >> 1);
      const float pin = s.pin[i], own = s.tb[w4];
      const bool direct = !(fabsf(own) <= 80.f);
      wait(&bar.s_full[it & 1], it >> 1);
      ptx::tc_fence_after();
      // blocks from the diagonal back; `between` sums the log-decays from the
      // block's end to row i
      float between = pin - own;
#pragma unroll 1
      for (int b = w4; b >= 0; --b) {
        const uint32_t at = tmem + ST_S + 128 * (it & 1) + 32 * b + c + lanes;
        uint32_t r[16];
        tmem_ld16_async(at, r);
        const float e = __expf(between);
        const float ee[2] = {e, e};
        between = b == w4 ? pin : between + s.tb[b];
        float v[16];
#pragma unroll
        for (int j = 0; j < 16; j += 4) {
          const float4 f = *reinterpret_cast<const float4 *>(&s.f[32 * b + c + j]);
          v[j] = f.x; v[j + 1] = f.y; v[j + 2] = f.z; v[j + 3] = f.w;
          mul_row<2>(v + j, v + j, ee);
          mul_row<2>(v + j + 2, v + j + 2, ee);
        }
        if (b == w4 && direct) {
          const float step =
              i < n ? ssm_step(p, q.b * p.dtb + (int64_t)(q.lo + it * ST_Q + i) * p.dts, h,
                               p.dt_bias ? p.dt_bias[h] : 0.f)
                    : 0.f;
          // log-decays up to row i, each rounded to 2^-19, so that their differences are
          // exact; e^-104 is zero in float32, and 32 of it stay below 2^31
          int sum = __float2int_rn(fmaxf(-expf(p.A_log[h]) * step, -104.f) * 524288.f);
#pragma unroll
          for (int o = 1; o < 32; o <<= 1) {
            const int u = __shfl_up_sync(~0u, sum, o);
            if (lane >= o) sum += u;
          }
#pragma unroll
          for (int j = 0; j < 16; ++j)
            v[j] = __expf((float)(sum - __shfl_sync(~0u, sum, c + j)) * 0x1p-19f) *
                   __shfl_sync(~0u, step, c + j);
        }
        tmem_wait_ld();
        pin_regs<16>(r);
#pragma unroll
        for (int j = 0; j < 16; j += 2) {
          const float x[2] = {__uint_as_float(r[j]), __uint_as_float(r[j + 1])};
          mul_row<2>(v + j, v + j, x);
        }
        if (b == w4 || n < ST_Q) {  // past the diagonal, past the sequence's end
          const int most = min(b == w4 ? lane : 31, n - 1 - 32 * b) - c;
          const int diag = b == w4 ? lane - c : -1;
#pragma unroll
          for (int j = 0; j < 16; ++j) {
            v[j] = j <= most ? v[j] : 0.f;
            if (j == diag) v[j] += skip;
          }
        }
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          r[j] = pack2(v[2 * j], v[2 * j + 1]);
          float d[2] = {low(r[j]), high(r[j])};
          sub_row<2>(d, v + 2 * j, d);
          r[8 + j] = pack2(d[0], d[1]);
        }
        tmem_st16(at, r);
      }
      const uint32_t zero[16] = {};
#pragma unroll 1
      for (int b = w4 + 1; b < 4; ++b) tmem_st16(tmem + ST_S + 128 * (it & 1) + 32 * b + c + lanes, zero);
      tmem_wait_st();
      ptx::tc_fence_before();
      arrive(&bar.ready[it & 1]);
      arrive(&bar.sc_free[it & 1]);
    }
  } else if (warp < ST_W_STATE) {
    // ---------------- output
    const int i = 32 * (warp & 3) + lane, c0 = 32 * ((warp - ST_W_OUT) >> 2);
    unsigned char *yt = sm + L::Y;
    // z comes straight to registers, 8 columns on their way (from L2, where the
    // loads ask for them) while the gate of the 8 before waits for y
    Row<__nv_bfloat16, 8> z;
    float gate[8];
    auto ask = [&](int it, int c) {
      const int64_t t = q.lo + (int64_t)it * ST_Q + i;
      if (t < q.hi && c < width)
        z.load(static_cast<const __nv_bfloat16 *>(p.z) + q.b * p.zb + t * p.zs + (int64_t)h * V +
               v0 + c);
    };
#pragma unroll
    for (int j = 0; j < 8; ++j) gate[j] = 1.f;
    z.zero();
    if (!STATES && p.z) {
      ask(0, c0);
      z.widen(gate);
      silu_row<8>(gate, gate);
      ask(0, c0 + 8);
    }
#pragma unroll 1
    for (int it = 0; it < (STATES ? 0 : nch) && going(); ++it) {
      const int n = tokens_of(it);
      const bool whole = n == ST_Q && !p.y_f32;
      wait(&bar.y_full[it & 1], it >> 1);
      ptx::tc_fence_after();
      const bool poisoned = it * ST_Q + i >= *const_cast<volatile int *>(&bad.any);
#pragma unroll 1
      for (int c = c0; c < c0 + 32; c += 8) {
        uint32_t acc[8];
        tmem_ld8_async(tmem + ST_Y + 64 * (it & 1) + c + lanes, acc);
        if (c == c0 && it > 0) wait(&bar.y_sent, it - 1);
        tmem_wait_ld();
        pin_regs<8>(acc);
        if (c == c0 + 24) {
          ptx::tc_fence_before();
          arrive(&bar.y_read[it & 1]);
        }
        float y[8];
#pragma unroll
        for (int j = 0; j < 8; j += 2) {
          const float x[2] = {__uint_as_float(acc[j]), __uint_as_float(acc[j + 1])};
          mul_row<2>(y + j, gate + j, x);
        }
        if (poisoned) {
#pragma unroll
          for (int j = 0; j < 8; ++j)
            if (it * ST_Q + i >= bad.first[c + j]) y[j] = __uint_as_float(0x7fffffffu);
        }
        Row<__nv_bfloat16, 8> out;
        out.round(y);
        if (whole) {
          out.store(reinterpret_cast<__nv_bfloat16 *>(yt + swz(i, c / 8)));
        } else if (i < n && c < width) {
          const int64_t at = q.b * p.yb + (q.lo + it * ST_Q + i) * p.ys + (int64_t)h * V + v0 + c;
          if (!p.y_f32) {
            out.store(static_cast<__nv_bfloat16 *>(p.y) + at);
          } else {
#pragma unroll
            for (int j = 0; j < 8; j += 4)
              *reinterpret_cast<float4 *>(static_cast<float *>(p.y) + at + j) =
                  make_float4(y[j], y[j + 1], y[j + 2], y[j + 3]);
          }
        }
        if (c == c0 + 24) {
          ptx::fence_proxy_async_smem();
          arrive(&bar.staged);
        }
        if (p.z) {
          z.widen(gate);
          silu_row<8>(gate, gate);
          const bool later = c >= c0 + 16;
          ask(it + later, c + (later ? -16 : 16));
        }
      }
    }
  } else if (warp < ST_W_W) {
    // ---------------- state: key k, columns v .. v + 31
    regs_up<ST_R_STATE>();
    const int k = 32 * (warp & 3) + lane, v = 32 * ((warp - ST_W_STATE) >> 2);
    const int cols = k < K ? min(32, width - v) : 0;
    const int64_t tile = (int64_t)V * K, at = (int64_t)(v0 + v) * K + k;
    float s[32];
#pragma unroll
    for (int j = 0; j < 32; ++j) s[j] = 0.f;
    auto add = [&](const float *src, float d) {
      src += at;
#pragma unroll
      for (int j = 0; j < 32; ++j, src += K) {
        if (j < cols) s[j] = fmaf(d, s[j], *src);
        if (j % 8 == 7) asm volatile("" ::: "memory");  // eight loads at a time
      }
    };
    if (!STATES) {
      if (p.h0) add(p.h0 + ((int64_t)q.n * p.H + h) * tile, 0.f);
#pragma unroll 1
      for (int i = q.first; i < item; ++i)
        add(p.seg_state + ((int64_t)i * p.H + h) * tile,
            expf(p.seg_decay[(int64_t)i * p.H + h]));
    }
    unsigned char *img = sm + L::H;
#pragma unroll 1
    for (int it = 0; it < nch && going(); ++it) {
      if (!STATES) {
        // C h^T of the chunk before has read the pieces: it ran before the
        // product whose result the state now holds
        if (k < 64 * KH) {
#pragma unroll
          for (int c = 0; c < 4; ++c) {
            uint32_t hi[4], lo[4];
#pragma unroll
            for (int j = 0; j < 4; ++j) {
              hi[j] = pack2(s[8 * c + 2 * j], s[8 * c + 2 * j + 1]);
              float d[2] = {low(hi[j]), high(hi[j])};
              sub_row<2>(d, s + 8 * c + 2 * j, d);
              lo[j] = pack2(d[0], d[1]);
            }
            *reinterpret_cast<uint4 *>(img + swz(k, v / 8 + c)) = make_uint4(hi[0], hi[1], hi[2], hi[3]);
            *reinterpret_cast<uint4 *>(img + ST_TILE + swz(k, v / 8 + c)) =
                make_uint4(lo[0], lo[1], lo[2], lo[3]);
          }
        }
        ptx::fence_proxy_async_smem();
        arrive(&bar.h_full);
      }
      wait(&bar.sc_full[it & 1], it >> 1);
      const float d = expf(sc[it & 1].total);
      const float dd[2] = {d, d};
      if (STATES) {
        arrive(&bar.sc_free[it & 1]);
      } else {
        float G = sc[it & 1].pin[k];
#pragma unroll
        for (int b = 0; b < 3; ++b) G += b < (warp & 3) ? sc[it & 1].tb[b] : 0.f;
        arrive(&bar.sc_free[it & 1]);
        const float e = __expf(G), ee[2] = {e, e};
        wait(&bar.off_full, it);
        ptx::tc_fence_after();
#pragma unroll 1
        for (int c = v; c < v + 32; c += 8) {
          uint32_t a[8];
          const uint32_t at = tmem + ST_Y + 64 * (it & 1) + c + lanes;
          tmem_ld8_async(at, a);
          tmem_wait_ld();
          pin_regs<8>(a);
#pragma unroll
          for (int j = 0; j < 8; j += 2) {
            float x[2] = {__uint_as_float(a[j]), __uint_as_float(a[j + 1])};
            mul_row<2>(x, x, ee);
            a[j] = __float_as_uint(x[0]);
            a[j + 1] = __float_as_uint(x[1]);
          }
          tmem_st8(at, a);
        }
        tmem_wait_st();
        ptx::tc_fence_before();
        arrive(&bar.ready[it & 1]);
      }
      wait(&bar.dh_full, it);
      ptx::tc_fence_after();
#pragma unroll
      for (int c = 0; c < 32; c += 8) {
        uint32_t a[8], b[8];
        tmem_ld8_async(tmem + ST_DH + v + c + lanes, a);
        tmem_ld8_async(tmem + ST_DH + 64 + v + c + lanes, b);
        tmem_wait_ld();
        pin_regs<8>(a);
        pin_regs<8>(b);
#pragma unroll
        for (int j = 0; j < 8; j += 2) {
          float x[2] = {__uint_as_float(b[j]), __uint_as_float(b[j + 1])};
          const float u[2] = {__uint_as_float(a[j]), __uint_as_float(a[j + 1])};
          add_row<2>(x, x, u);
          fma_row<2>(x, dd, s + c + j);
          s[c + j] = x[0];
          s[c + j + 1] = x[1];
        }
      }
      ptx::tc_fence_before();
      arrive(&bar.dh_free);
    }
    float *dst = STATES               ? p.seg_state + ((int64_t)item * p.H + h) * tile
                 : q.last && p.ht != nullptr ? p.ht + ((int64_t)q.n * p.H + h) * tile
                                             : nullptr;
    if (dst && ok) {
      dst += at;
#pragma unroll
      for (int j = 0; j < 32; ++j, dst += K)
        if (j < cols) *dst = s[j];
    }
  } else if (warp < ST_W_LOAD) {
    // ---------------- W: row j of the chunk
    regs_down<ST_R_W>();
    const int j = tid - 32 * ST_W_W;
    unsigned char *img = sm + L::W;
#pragma unroll 1
    for (int it = 0; it < nch && going(); ++it) {
      unsigned char *xt = sm + L::X + (it & 1) * ST_TILE, *bt = sm + L::B + (it & 1) * KH * ST_TILE;
      const int n = tokens_of(it);
      wait(&bar.sc_full[it & 1], it >> 1);
      const float w = sc[it & 1].f[j] * sc[it & 1].sfx[j >> 5];
      arrive(&bar.sc_free[it & 1]);
      wait(&bar.x_full[it & 1], it >> 1);
      if (n < ST_Q) wait(&bar.b_full[it & 1], it >> 1);
      if (it > 0) wait(&bar.dh_full, it - 1);  // the product before has read W
      if (j < n) {
        const float ww[2] = {w, w};
        // NaNs once an element of the row is not finite: its last piece is NaN
        __nv_bfloat162 odd = __floats2bfloat162_rn(0.f, 0.f);
#pragma unroll 1
        for (int c = 0; c < 8; ++c) {
          const uint4 u = *reinterpret_cast<const uint4 *>(xt + swz(j, c));
          const uint32_t x[4] = {u.x, u.y, u.z, u.w};
          uint32_t a[4], b[4], e[4];
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            // p = hi + mid + lo, each the bf16 nearest to what is left
            float v[2] = {low(x[k]), high(x[k])}, d[2];
            mul_row<2>(v, v, ww);
            a[k] = pack2(v[0], v[1]);
            d[0] = low(a[k]); d[1] = high(a[k]);
            sub_row<2>(v, v, d);
            b[k] = pack2(v[0], v[1]);
            d[0] = low(b[k]); d[1] = high(b[k]);
            sub_row<2>(v, v, d);
            e[k] = pack2(v[0], v[1]);
            odd = __hfma2(*reinterpret_cast<const __nv_bfloat162 *>(&e[k]),
                          __floats2bfloat162_rn(0.f, 0.f), odd);
          }
          *reinterpret_cast<uint4 *>(img + swz(j, c)) = make_uint4(a[0], a[1], a[2], a[3]);
          *reinterpret_cast<uint4 *>(img + ST_TILE + swz(j, c)) = make_uint4(b[0], b[1], b[2], b[3]);
          *reinterpret_cast<uint4 *>(img + 2 * ST_TILE + swz(j, c)) =
              make_uint4(e[0], e[1], e[2], e[3]);
        }
        if (!__hbeq2(odd, odd)) {
#pragma unroll 1
          for (int c = 0; c < ST_VT; ++c) {
            const uint32_t at = swz(j, c / 8) + 2 * (c % 8);
            auto half = [&](unsigned char *tile) { return reinterpret_cast<uint16_t *>(tile + at); };
            auto finite = [](const uint16_t *v) { return (*v & 0x7f80) != 0x7f80; };
            // an infinite first piece is the whole value: Inf - Inf left no others
            if (!finite(half(img))) *half(img + ST_TILE) = *half(img + 2 * ST_TILE) = 0;
            if (STATES || finite(half(xt))) continue;
            *half(xt) = 0;
            atomicMin(&bad.first[c], it * ST_Q + j);
            atomicMin(&bad.any, it * ST_Q + j);
          }
        }
      } else {
        // past the sequence's end: what the loads brought is another sequence's
        const uint4 zero = make_uint4(0, 0, 0, 0);
#pragma unroll 1
        for (int c = 0; c < 8; ++c) {
#pragma unroll
          for (int b = 0; b < 3; ++b) *reinterpret_cast<uint4 *>(img + b * ST_TILE + swz(j, c)) = zero;
          *reinterpret_cast<uint4 *>(xt + swz(j, c)) = zero;
#pragma unroll
          for (int b = 0; b < KH; ++b)
            *reinterpret_cast<uint4 *>(bt + b * ST_TILE + swz(j, c)) = zero;
        }
      }
      ptx::fence_proxy_async_smem();
      arrive(&bar.w_full);
    }
  } else if (warp == ST_W_LOAD) {
    // ---------------- loads
    regs_down<ST_R_REST>();
    if (lane == 0) {
      ptx::prefetch_tmap(&tm_x);
      ptx::prefetch_tmap(&tm_b);
      if (!STATES) ptx::prefetch_tmap(&tm_c);
    }
    int xs = 0, bms = 0;  // tiles asked for
#pragma unroll 1
    for (int it = 0; it < nch && going(); ++it) {
      const int bs = it & 1, t = q.lo + it * ST_Q;
      // one copy a lane: the copies of one thread complete one after another
      if (it >= 2) wait(&bar.b_free[bs], (it >> 1) - 1);
      if (!going()) break;
      if (lane == 0) ptx::mbar_arrive_expect_tx(&bar.b_full[bs], KH * ST_TILE);
      __syncwarp();
      if (lane >= 1 && lane <= KH)
        tma_load_4d(sm + L::B + (bs * KH + lane - 1) * ST_TILE, &tm_b, 64 * (lane - 1), g, t, q.b,
                    &bar.b_full[bs]);
      ++bms;
      if (it >= 2) wait(&bar.x_free[bs], (it >> 1) - 1);
      if (!going()) break;
      if (lane == 0) {
        ptx::mbar_arrive_expect_tx(&bar.x_full[bs], ST_TILE);
        tma_load_4d(sm + L::X + bs * ST_TILE, &tm_x, v0, h, t, q.b, &bar.x_full[bs]);
        if (it + 2 < nch) tma_prefetch_4d(&tm_x, v0, h, t + 2 * ST_Q, q.b);
      }
      ++xs;
      if (!STATES) {
        if (it >= 1) wait(&bar.off_full, it - 1);  // C h^T, the last to read C
        if (!going()) break;
        if (lane == 0) ptx::mbar_arrive_expect_tx(&bar.b_full[bs], KH * ST_TILE);
        __syncwarp();
        if (lane > KH && lane <= 2 * KH) {
          const int half = lane - 1 - KH;
          tma_load_4d(sm + L::C + half * ST_TILE, &tm_c, 64 * half, g, t, q.b,
                      &bar.b_full[bs]);
          if (it + 1 < nch) tma_prefetch_4d(&tm_c, 64 * half, g, t + ST_Q, q.b);
        }
        if (p.z && lane == 0 && it + 1 < nch) tma_prefetch_4d(&tm_z, v0, h, t + ST_Q, q.b);
      }
    }
    // the last copies land before the block ends, whoever else waits for them
    for (int k = max(0, xs - 2); k < xs; ++k) drain(&bar.x_full[k & 1], k >> 1);
    for (int k = max(0, bms - 2); k < bms; ++k) drain(&bar.b_full[k & 1], k >> 1);
  } else if (warp == ST_W_MMA) {
    // ---------------- MMA
    regs_down<ST_R_REST>();
    const uint32_t id_s = ptx::idesc_bf16(128, 128, 0, 0);    // C, B K-major
    const uint32_t id_y = ptx::idesc_bf16(128, 64, 0, 1);     // C or M, h or x MN-major
    const uint32_t id_dh2 = ptx::idesc_bf16(128, 128, 1, 1);  // B, two pieces of W MN-major
    const uint32_t id_dh1 = ptx::idesc_bf16(128, 64, 1, 1);
    const uint32_t one = elect_one();
    const uint32_t dc = sw128(sm + L::C, 16), dh = sw128(sm + L::H, ST_TILE);
    const uint32_t dw = sw128(sm + L::W, ST_TILE);
    auto b_of = [&](int it) { return (uint32_t)(L::B + (it & 1) * KH * ST_TILE); };
    // (S goes where M was two chunks before: M X of that chunk is behind the
    // C h^T whose scaled rows `ready` has announced since)
    auto scores = [&](int it) {
      const uint32_t db = sw128(sm + b_of(it), 16), d = tmem + ST_S + 128 * (it & 1);
      wait(&bar.b_full[it & 1], it >> 1);
      if (!going()) return;
      ptx::tc_fence_after();
#pragma unroll 1
      for (int half = 0; half < KH; ++half)
#pragma unroll 2
        for (int ks = 0; ks < 4; ++ks)
          mma_ss(one, d, ahead(dc, half * ST_TILE + ks * 32), ahead(db, half * ST_TILE + ks * 32),
                 id_s, half + ks > 0);
      commit(one, &bar.s_full[it & 1]);
    };
    auto carried = [&](int it) {  // C h^T
      wait(&bar.h_full, it);
      if (it > 1) wait(&bar.y_read[it & 1], (it >> 1) - 1);
      if (!going()) return;
      ptx::tc_fence_after();
      const uint32_t d = tmem + ST_Y + 64 * (it & 1);
#pragma unroll 1
      for (int half = 0; half < KH; ++half)
#pragma unroll 2
        for (int ks = 0; ks < 4; ++ks) {
          const uint32_t a = ahead(dc, half * ST_TILE + ks * 32), b = ahead(dh, (4 * half + ks) * 2048);
          mma_ss(one, d, a, b, id_y, half + ks > 0);
          mma_ss(one, d, a, ahead(b, ST_TILE), id_y, 1);
        }
      commit(one, &bar.off_full);
    };
    if (!STATES && nch > 0) {
      scores(0);
      carried(0);
    }
#pragma unroll 1
    for (int it = 0; it < nch && going(); ++it) {
      // with one half of keys the product's upper 64 rows are of the tile after
      // B, and are not read
      const uint32_t db = sw128(sm + b_of(it), ST_TILE);
      wait(&bar.w_full, it);
      if (STATES) {  // else the scores' b_full and C h^T's h_full said so
        wait(&bar.b_full[it & 1], it >> 1);
        if (it > 0) wait(&bar.dh_free, it - 1);
      }
      if (!going()) break;
      ptx::tc_fence_after();
#pragma unroll 1
      for (int k4 = 0; k4 < 8; k4 += 2)
#pragma unroll
        for (int ks = 0; ks < 2; ++ks) {
          const uint32_t a = ahead(db, (k4 + ks) * 2048), b = ahead(dw, (k4 + ks) * 2048);
          mma_ss(one, tmem + ST_DH, a, b, id_dh2, k4 + ks > 0);
          mma_ss(one, tmem + ST_DH + 64, a, ahead(b, 2 * ST_TILE), id_dh1, 1);
        }
      commit(one, &bar.dh_full);
      commit(one, &bar.b_free[it & 1]);
      if (STATES) {
        commit(one, &bar.x_free[it & 1]);
        continue;
      }
      wait(&bar.ready[it & 1], it >> 1);
      if (!going()) break;
      if (it + 1 < nch) scores(it + 1);
      ptx::tc_fence_after();
      const uint32_t dx = sw128(sm + L::X + (it & 1) * ST_TILE, ST_TILE);
      const uint32_t dm = tmem + ST_S + 128 * (it & 1), dy = tmem + ST_Y + 64 * (it & 1);
#pragma unroll 1
      for (int k4 = 0; k4 < 16; k4 += 2)
#pragma unroll
        for (int ks = 0; ks < 2; ++ks)
          mma_ts(one, dy, dm + 8 * (k4 + ks), ahead(dx, ((k4 + ks) >> 1) * 2048), id_y, 1);
      commit(one, &bar.y_full[it & 1]);
      commit(one, &bar.x_free[it & 1]);
      if (it + 1 < nch) carried(it + 1);
    }
    commit(one, &bar.drained);
    drain(&bar.drained, 0);
  } else if (warp == ST_W_SCALARS) {
    // ---------------- scalars
    regs_down<ST_R_REST>();
    const float a = -expf(p.A_log[h]), bias = p.dt_bias ? p.dt_bias[h] : 0.f;
    float sum = 0.f;  // of the whole segment's log-decays
    auto fetch = [&](int it, uint32_t (&raw)[4]) {  // dt's bits, on their way
#pragma unroll
      for (int b = 0; b < 4; ++b) {
        const int64_t t = q.lo + (int64_t)it * ST_Q + 32 * b + lane;
        raw[b] = 0;
        if (t < q.hi) {
          const int64_t at = q.b * p.dtb + t * p.dts + h;
          if (p.dt_f32)
            raw[b] = static_cast<const uint32_t *>(p.dt)[at];
          else
            raw[b] = static_cast<const uint16_t *>(p.dt)[at];
        }
      }
    };
    auto put = [&](int it, const uint32_t (&raw)[4]) {
      StScalars &s = sc[it & 1];
      // the four blocks side by side: their sums are long chains of shuffles
      float step[4], before[4], after[4];  // sums up to and from this token
#pragma unroll
      for (int b = 0; b < 4; ++b) {
        const float v = __uint_as_float(p.dt_f32 ? raw[b] : raw[b] << 16) + bias;
        const float soft = log1pf(expf(fminf(v, 20.f)));
        step[b] = !p.softplus || !(v <= 20.f) ? v : soft;
        if (q.lo + it * ST_Q + 32 * b + lane >= q.hi) step[b] = 0.f;
        before[b] = after[b] = a * step[b];
      }
#pragma unroll 1
      for (int o = 1; o < 32; o <<= 1) {
#pragma unroll
        for (int b = 0; b < 4; ++b) {
          const float u = __shfl_up_sync(~0u, before[b], o), d = __shfl_down_sync(~0u, after[b], o);
          if (lane >= o) before[b] += u;
          if (lane + o < 32) after[b] += d;
        }
      }
      float tail = 0.f;
#pragma unroll
      for (int b = 3; b >= 0; --b) {
        const float all = __shfl_sync(~0u, before[b], 31);
        const float rest = __shfl_down_sync(~0u, after[b], 1);
        s.pin[32 * b + lane] = before[b];
        s.f[32 * b + lane] = step[b] * expf(lane < 31 ? rest : 0.f);
        if (lane == 0) {
          s.tb[b] = all;
          s.sfx[b] = expf(tail);
        }
        tail += all;
      }
      if (lane == 0) s.total = tail;
      sum += tail;
      arrive(&bar.sc_full[it & 1]);
    };
    uint32_t raw[4];
    fetch(0, raw);
#pragma unroll 1
    for (int it = 0; it < nch && going(); ++it) {
      uint32_t next[4];
      fetch(it + 1, next);
      if (it >= 2) wait(&bar.sc_free[it & 1], (it >> 1) - 1);
      put(it, raw);
#pragma unroll
      for (int b = 0; b < 4; ++b) raw[b] = next[b];
    }
    if (STATES && lane == 0 && v0 == 0 && ok) p.seg_decay[(int64_t)item * p.H + h] = sum;
  } else if (!STATES) {
    // ---------------- store
    regs_down<ST_R_REST>();
#pragma unroll 1
    for (int it = 0; it < nch && going(); ++it) {
      wait(&bar.staged, it);
      if (!going()) break;
      if (lane == 0) {
        if (tokens_of(it) == ST_Q && !p.y_f32) {
          tma_store_4d(&tm_y, v0, h, q.lo + it * ST_Q, q.b, sm + L::Y);
          ptx::bulk_commit();
          ptx::bulk_wait_read<0>();
        }
        ptx::mbar_arrive(&bar.y_sent);
      }
      __syncwarp();
    }
    if (lane == 0) ptx::bulk_wait<0>();
  } else {
    regs_down<ST_R_REST>();
  }
  if (!ok && lane == 0) record_error(p.err, GDN_ERR_TIMEOUT);
  ptx::tc_fence_before();
  __syncthreads();
  if (warp == 0) ptx::tmem_dealloc<512>(tmem);
}

// [batch][token][heads][dim] bf16 with strides between tokens and batch rows;
// boxes of 64 columns of one head over 128 tokens in 128-byte swizzled rows.
bool token_map(CUtensorMap *m, const void *base, int dim, int heads, int T, int B, int64_t stride,
               int64_t batch_stride) {
  const auto fn = tensor_map_encoder();
  if (!fn) return false;
  const cuuint64_t gdim[4] = {(cuuint64_t)dim, (cuuint64_t)heads, (cuuint64_t)T, (cuuint64_t)B};
  const cuuint64_t gstride[3] = {(cuuint64_t)dim * 2, (cuuint64_t)stride * 2,
                                 (cuuint64_t)(B > 1 ? batch_stride : stride) * 2};
  const cuuint32_t box[4] = {ST_VT, 1, ST_Q, 1}, step[4] = {1, 1, 1, 1};
  return fn(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 4, const_cast<void *>(base), gdim, gstride, box,
            step, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
            CU_TENSOR_MAP_L2_PROMOTION_L2_128B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

template <int KH>
cudaError_t launch(const SsmParams &p, cudaStream_t stream) {
  CUtensorMap x, b, c, z, y;
  if (!token_map(&x, p.x, p.V, p.H, p.T, p.B, p.xs, p.xb) ||
      !token_map(&b, p.Bm, p.K, p.Hg, p.T, p.B, p.bs, p.bb) ||
      !token_map(&c, p.Cm, p.K, p.Hg, p.T, p.B, p.cs, p.cb))
    return cudaErrorInvalidValue;
  z = y = x;  // not used without a gate, or for a float32 y
  if (p.z && !token_map(&z, p.z, p.V, p.H, p.T, p.B, p.zs, p.zb)) return cudaErrorInvalidValue;
  if (!p.y_f32 && !token_map(&y, p.y, p.V, p.H, p.T, p.B, p.ys, p.yb)) return cudaErrorInvalidValue;
  constexpr int bytes = StLayout<KH>::BYTES;
  const dim3 grid((unsigned)(p.H * ((p.V + ST_VT - 1) / ST_VT)), (unsigned)p.items);
  if (p.seg_state) {
    const cudaError_t e = cudaFuncSetAttribute(
        ssm_tc_kernel<KH, true>, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
    if (e != cudaSuccess) return e;
    ssm_tc_kernel<KH, true><<<grid, ST_THREADS, bytes, stream>>>(x, b, c, z, y, p);
  }
  const cudaError_t e = cudaFuncSetAttribute(
      ssm_tc_kernel<KH, false>, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
  if (e != cudaSuccess) return e;
  ssm_tc_kernel<KH, false><<<grid, ST_THREADS, bytes, stream>>>(x, b, c, z, y, p);
  return cudaGetLastError();
}

bool even(const void *base, int64_t stride, int64_t batch_stride) {
  return (reinterpret_cast<uintptr_t>(base) & 15u) == 0 && stride % 8 == 0 && batch_stride % 8 == 0;
}

}  // namespace

bool ssm_tc_supported(const SsmParams &p, bool bf16) {
  // rows of 16-byte pieces throughout; one launch index counts (head, V tile)
  return bf16 && p.T > 0 && p.K % 8 == 0 && p.V % 8 == 0 && p.K <= 128 &&
         p.items <= MAX_GRID_YZ && even(p.x, p.xs, p.xb) && even(p.Bm, p.bs, p.bb) &&
         even(p.Cm, p.cs, p.cb) && (p.z == nullptr || even(p.z, p.zs, p.zb)) &&
         even(p.y, p.ys, p.yb);
}

cudaError_t launch_ssm_tc(const SsmParams &p, cudaStream_t stream) {
  return p.K <= 64 ? launch<1>(p, stream) : launch<2>(p, stream);
}

}  // namespace gdn
