// Matrix fragments, images and the workspace of the gated delta rule's gradient on the tensor
// cores, shared by delta_bwd_tc.cu (T and P of every chunk), delta_bwd_walk.cu (the states and
// their gradients, chunk after chunk) and delta_bwd_inputs.cu (the inputs' gradients).
// delta_bwd.h has the formulas.
//
// Where products stand between element-wise gates, masks and sums, accumulators stay in
// registers (warp-level matrix instructions) instead of passing through tensor memory between
// each two of them; what is plain contraction runs on tcgen05.  q, k, v and do are bfloat16 and
// exact; what is float32 (T, P, the states h and their gradients D, the corrected values n and
// dr) enters as a pair of bfloat16 pieces, hi + lo, with the products hi hi + hi lo + lo hi (lo lo
// where dbeta and dg add many of them up): off by 2^-17 of each value at most, so that the float32 results (dg, dbeta, dh0) are not
// bound by bfloat16.  Accumulation is float32.
//
// Images lie in shared memory as rows of 64, 128 or 256 bytes whose 16-byte pieces are
// exchanged by row (`at`), so that matrix loads touch every bank once; the workspace holds
// the same images, so that the next kernel fetches them by straight copies.
#pragma once

#include "delta_bwd.h"
#include "gdn_common.cuh"
#include "ptx.cuh"
#include "rows.cuh"

namespace gdn {

using bf16 = __nv_bfloat16;

constexpr int Q = 64;    // tokens of a chunk
constexpr int VT = 32;   // value columns of a tile

// Place of (row, col) in an image with rows of COLS elements (72 or 136: rows of 64 or 128 that
// lie a piece further apart instead).
template <int COLS>
__device__ __forceinline__ int at(int row, int col) {
  if constexpr (COLS % 16 == 8) return row * COLS + col;
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

// A chunk and head in the workspace (bytes; KP = K rounded up to 64 or 128): G, beta, e^G and
// e^(G_L - G) of its tokens (past its end G = G_L and beta = 0), then matrices, each hi then
// lo: T, P and A without beta as images; by value tiles n, dr [32][64] and h, D [32][KP], value columns first, as
// 8 x 8 tiles of 128 bytes (a warp holds such a tile as a word a lane, in this order).  What G's
// rounding left lies in the first rows of T's upper right block, which is zero and which no walk
// reads.
template <int KP>
struct Block {
  static constexpr int SC = 4 * Q * 4, SQUARE = 2 * Q * Q * 2, ROWS = 2 * Q * VT * 2,
                       STATE = 2 * KP * VT * 2;
  unsigned char *base;
  int tiles;
  __device__ Block(const DeltaBwdParams &p, int64_t chunk, int head)
      : base(p.blocks + (chunk * p.H + head) * p.block), tiles((p.V + VT - 1) / VT) {}
  __device__ float *sc() const { return reinterpret_cast<float *>(base); }
  __device__ unsigned char *T() const { return base + SC; }
  // where token i's rest lies in T's first image
  static __device__ __forceinline__ int rest_at(int i) { return at<64>(i >> 3, 48 + 2 * (i & 7)); }
  __device__ float rest(int i) const {
    return *reinterpret_cast<const float *>(reinterpret_cast<const bf16 *>(T()) + rest_at(i));
  }
  __device__ unsigned char *P() const { return base + SC + SQUARE; }
  __device__ unsigned char *n(int v) const { return base + SC + 3 * SQUARE + v * ROWS; }
  __device__ unsigned char *dr(int v) const { return n(tiles) + v * ROWS; }
  __device__ unsigned char *h(int v) const { return dr(tiles) + v * STATE; }
  __device__ unsigned char *D(int v) const { return h(tiles) + v * STATE; }
  static int64_t bytes(int tiles) {
    return SC + 3 * SQUARE + (int64_t)tiles * 2 * (ROWS + STATE);
  }
};

// A straight copy from shared memory to the workspace, by all threads.
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
  for (int i = threadIdx.x % THREADS; i < Q * COLS / 8; i += THREADS) {
    const int row = i / (COLS / 8), col = i % (COLS / 8) * 8;
    const bool ok = row < ch.len && c0 + col < D;
    ptx::cp_async16(to + at<COLS>(row, col), ok ? from + row * stride + c0 + col : from, ok);
  }
}

// x and y as two words, the upper and the lower pieces.
__device__ __forceinline__ void split(float x, float y, uint32_t &hi, uint32_t &lo) {
  const __nv_bfloat162 h = __floats2bfloat162_rn(x, y);
  const float2 f = __bfloat1622float2(h);
  const __nv_bfloat162 l = __floats2bfloat162_rn(x - f.x, y - f.y);
  hi = *reinterpret_cast<const uint32_t *>(&h);
  lo = *reinterpret_cast<const uint32_t *>(&l);
}

// Most blocks of the kernel of the inputs' gradients (each has scratch of its own).
constexpr int DELTA_MAX_BLOCKS = 256;

cudaError_t launch_delta_inputs(const DeltaBwdParams &p, cudaStream_t stream);
cudaError_t launch_delta_walks(const DeltaBwdParams &p, cudaStream_t stream);

}  // namespace gdn
