// Pieces of token rows in registers, and the checks of packed sequences, shared
// by the short convolution and the state space scan.
#pragma once

#include "gdn_common.cuh"

namespace gdn {

// VEC consecutive elements of a row as raw words, so that rows can be on the
// way without being widened.
template <typename T, int VEC>
struct Row {
  static constexpr int BYTES = VEC * (int)sizeof(T);
  static constexpr int WORDS = BYTES >= 4 ? BYTES / 4 : 1;
  uint32_t w[WORDS];

  __device__ __forceinline__ void zero() {
#pragma unroll
    for (int i = 0; i < WORDS; ++i) w[i] = 0;
  }
  __device__ __forceinline__ void load(const T *p) {
    if constexpr (BYTES == 16) {
      const uint4 u = *reinterpret_cast<const uint4 *>(p);
      w[0] = u.x; w[1] = u.y; w[2] = u.z; w[3] = u.w;
    } else if constexpr (BYTES == 8) {
      const uint2 u = *reinterpret_cast<const uint2 *>(p);
      w[0] = u.x; w[1] = u.y;
    } else if constexpr (BYTES == 4) {
      w[0] = *reinterpret_cast<const uint32_t *>(p);
    } else {
      w[0] = *reinterpret_cast<const uint16_t *>(p);
    }
  }
  __device__ __forceinline__ void store(T *p) const {
    if constexpr (BYTES == 16) {
      *reinterpret_cast<uint4 *>(p) = make_uint4(w[0], w[1], w[2], w[3]);
    } else if constexpr (BYTES == 8) {
      *reinterpret_cast<uint2 *>(p) = make_uint2(w[0], w[1]);
    } else if constexpr (BYTES == 4) {
      *reinterpret_cast<uint32_t *>(p) = w[0];
    } else {
      *reinterpret_cast<uint16_t *>(p) = (uint16_t)w[0];
    }
  }
  __device__ __forceinline__ void widen(float *f) const {
    if constexpr (sizeof(T) == 4) {
#pragma unroll
      for (int i = 0; i < VEC; ++i) f[i] = __uint_as_float(w[i]);
    } else if constexpr (VEC == 1) {
      f[0] = __uint_as_float(w[0] << 16);
    } else {
#pragma unroll
      for (int i = 0; i < VEC / 2; ++i) {
        f[2 * i] = __uint_as_float(w[i] << 16);
        f[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
      }
    }
  }
  __device__ __forceinline__ void round(const float *f) {
    if constexpr (sizeof(T) == 4) {
#pragma unroll
      for (int i = 0; i < VEC; ++i) w[i] = __float_as_uint(f[i]);
    } else if constexpr (VEC == 1) {
      w[0] = __bfloat16_as_ushort(__float2bfloat16_rn(f[0]));
    } else {
#pragma unroll
      for (int i = 0; i < VEC / 2; ++i) {
        const __nv_bfloat162 h = __floats2bfloat162_rn(f[2 * i], f[2 * i + 1]);
        w[i] = *reinterpret_cast<const uint32_t *>(&h);
      }
    }
  }
};

// acc[0..VEC) += a[0..VEC) * b[0..VEC), two lanes an instruction
template <int VEC>
__device__ __forceinline__ void fma_row(float *acc, const float *a, const float *b) {
  if constexpr (VEC == 1) {
    acc[0] = fmaf(a[0], b[0], acc[0]);
  } else {
#pragma unroll
    for (int i = 0; i < VEC; i += 2)
      asm("{\n\t.reg .b64 ra, rb, rc;\n\t"
          "mov.b64 ra, {%2, %3};\n\tmov.b64 rb, {%4, %5};\n\tmov.b64 rc, {%0, %1};\n\t"
          "fma.rn.f32x2 rc, ra, rb, rc;\n\tmov.b64 {%0, %1}, rc;\n\t}"
          : "+f"(acc[i]), "+f"(acc[i + 1])
          : "f"(a[i]), "f"(a[i + 1]), "f"(b[i]), "f"(b[i + 1]));
  }
}

// out = a * b + c
template <int VEC>
__device__ __forceinline__ void fma_rows(float *out, const float *a, const float *b,
                                         const float *c) {
  static_assert(VEC % 2 == 0, "pairs");
#pragma unroll
  for (int i = 0; i < VEC; i += 2)
    asm("{\n\t.reg .b64 ra, rb, rc;\n\t"
        "mov.b64 ra, {%2, %3};\n\tmov.b64 rb, {%4, %5};\n\tmov.b64 rc, {%6, %7};\n\t"
        "fma.rn.f32x2 rc, ra, rb, rc;\n\tmov.b64 {%0, %1}, rc;\n\t}"
        : "=f"(out[i]), "=f"(out[i + 1])
        : "f"(a[i]), "f"(a[i + 1]), "f"(b[i]), "f"(b[i + 1]), "f"(c[i]), "f"(c[i + 1]));
}

// out = a op b, pairs of lanes an instruction
#define GDN_ROW_OP(name, op)                                                           \
  template <int VEC>                                                                   \
  __device__ __forceinline__ void name(float *out, const float *a, const float *b) {   \
    static_assert(VEC % 2 == 0, "pairs");                                              \
    _Pragma("unroll") for (int i = 0; i < VEC; i += 2)                                 \
        asm("{\n\t.reg .b64 ra, rb;\n\t"                                               \
            "mov.b64 ra, {%2, %3};\n\tmov.b64 rb, {%4, %5};\n\t" op                    \
            ".rn.f32x2 ra, ra, rb;\n\tmov.b64 {%0, %1}, ra;\n\t}"                      \
            : "=f"(out[i]), "=f"(out[i + 1])                                           \
            : "f"(a[i]), "f"(a[i + 1]), "f"(b[i]), "f"(b[i + 1]));                     \
  }
GDN_ROW_OP(mul_row, "mul")
GDN_ROW_OP(add_row, "add")
GDN_ROW_OP(sub_row, "sub")
#undef GDN_ROW_OP

// p / (1 + e^-p); e^-p overflows to infinity below -88 and the quotient is 0
__device__ __forceinline__ float silu(float p) { return __fdividef(p, 1.f + __expf(-p)); }

// 1 / (1 + e^-z) of VEC values, and silu
template <int VEC>
__device__ __forceinline__ void sigmoid_row(float *out, const float *z) {
  const float k[2] = {-1.442695041f, -1.442695041f}, one[2] = {1.f, 1.f};
#pragma unroll
  for (int i = 0; i < VEC; i += 2) {
    float e[2];
    mul_row<2>(e, z + i, k);
#pragma unroll
    for (int j = 0; j < 2; ++j) asm("ex2.approx.ftz.f32 %0, %0;" : "+f"(e[j]));
    add_row<2>(e, e, one);
#pragma unroll
    for (int j = 0; j < 2; ++j) asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(out[i + j]) : "f"(e[j]));
  }
}
template <int VEC>
__device__ __forceinline__ void silu_row(float *out, const float *z) {
  float s[VEC];
  sigmoid_row<VEC>(s, z);
  mul_row<VEC>(out, z, s);
}

// log(1 + e^v), v itself above 20
__device__ __forceinline__ float softplus(float v) { return v > 20.f ? v : log1pf(expf(v)); }

// Whether cu_seqlens (NULL: nothing to check) rises from 0 to T; the whole
// block takes part.
__device__ __forceinline__ bool offsets_ok(const int32_t *cu, int N, int T, int *err) {
  if (cu == nullptr) return true;
  int bad = 0;
  const int threads = blockDim.x * blockDim.y, tid = threadIdx.y * blockDim.x + threadIdx.x;
  for (int n = tid; n <= N; n += threads) {
    const int v = cu[n];
    if (n == 0 && v != 0) bad = 1;
    if (n == N ? v != T : v > cu[n + 1]) bad = 1;
  }
  bad = __syncthreads_or(bad);
  if (bad && tid == 0) record_error(err, GDN_ERR_BAD_SEQLENS);
  return !bad;
}

}  // namespace gdn
