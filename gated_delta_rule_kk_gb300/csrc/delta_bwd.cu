// Gradient of the chunked gated delta rule: argument checks, workspace and the table of
// chunks of packed sequences.  delta_bwd.h has the formulas.
#include <math.h>

#include <algorithm>

#include "abi_check.h"
#include "delta_bwd.h"
#include "rows.cuh"

namespace gdn {
namespace {

// Sequences of about as many chunks, more of them first: four classes to a power of two.
constexpr int CLASSES = 128;
__device__ __forceinline__ int length_class(int chunks) {
  return chunks == 0 ? CLASSES - 1
                     : CLASSES - 2 - ((__float_as_int((float)chunks) >> 21) - (127 << 2));
}

// First chunk of every sequence, every chunk's sequence and the sequences by their lengths;
// with bad offsets first[N] = -1, and no kernel behind writes anything.  One block.  (The order
// among sequences of one class is any; it changes no result.)
__global__ void __launch_bounds__(1024) delta_table_kernel(DeltaBwdParams p) {
  __shared__ int sums[32], total, class_at[CLASSES];
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  if (!offsets_ok(p.cu, p.N, p.T, p.err)) {
    if (tid == 0) p.first[p.N] = -1;
    return;
  }
  if (tid == 0) total = 0;
  if (tid < CLASSES) class_at[tid] = 0;
  __syncthreads();
  for (int base = 0; base < p.N; base += 1024) {
    const int n = base + tid;
    int own = n < p.N ? (int)(((int64_t)p.cu[n + 1] - p.cu[n] + 63) / 64) : 0;
    int s = own;
    for (int o = 1; o < 32; o <<= 1) {
      const int v = __shfl_up_sync(~0u, s, o);
      if (lane >= o) s += v;
    }
    if (lane == 31) sums[warp] = s;
    __syncthreads();
    int before = total;
    for (int w = 0; w < warp; ++w) before += sums[w];
    if (n < p.N) {
      p.first[n] = before + s - own;
      atomicAdd(&class_at[length_class(own)], 1);
    }
    __syncthreads();
    if (tid == 1023) total = before + s;
    __syncthreads();
  }
  if (tid == 0) {
    p.first[p.N] = total;
    for (int c = 0, before = 0; c < CLASSES; ++c) {
      const int here = class_at[c];
      class_at[c] = before;
      before += here;
    }
  }
  __syncthreads();
  for (int n = tid; n < p.N; n += 1024)
    p.order[atomicAdd(&class_at[length_class(p.first[n + 1] - p.first[n])], 1)] = n;
  if (!bounds_ok(total <= p.chunks, p.err)) return;
  for (int c = tid; c < total; c += 1024) {  // the last sequence that begins at c or before
    int lo = 0, hi = p.N - 1;
    while (lo < hi) {
      const int mid = (lo + hi + 1) / 2;
      if (p.first[mid] <= c)
        lo = mid;
      else
        hi = mid - 1;
    }
    p.owner[c] = lo;
  }
}

// Without tokens the states' gradients pass through, where the offsets are all zero.
__global__ void __launch_bounds__(256) delta_none_kernel(DeltaBwdParams p, int64_t values) {
  if (!offsets_ok(p.cu, p.N, 0, p.err)) return;
  for (int64_t i = blockIdx.x * 256ll + threadIdx.x; i < values; i += gridDim.x * 256ll)
    p.dh0[i] = p.dht ? p.dht[i] : 0.f;
}

gdn_status_t check_args(const gdn_chunk_bwd_args &a, bool sizes_only) {
  CHECK_DTYPE(a.dtype, "dtype");
  CHECK_THAT(a.B >= 1 && a.T >= 0 && a.H >= 1 && a.Hg >= 1 && a.K >= 1 && a.V >= 1 && a.N >= 1,
             GDN_ERR_INVALID_ARG, "sizes must be positive (B=%d T=%d heads=%d/%d K=%d V=%d N=%d)",
             a.B, a.T, a.Hg, a.H, a.K, a.V, a.N);
  CHECK_THAT(a.H % a.Hg == 0, GDN_ERR_UNSUPPORTED, "H (%d) must be a multiple of Hg (%d)", a.H, a.Hg);
  CHECK_THAT(a.N <= 65535 && a.H <= 65535, GDN_ERR_UNSUPPORTED,
             "N (%d) and H (%d) must be at most 65535", a.N, a.H);
  CHECK_THAT(a.K <= 128, GDN_ERR_UNSUPPORTED, "K=%d exceeds 128", a.K);
  CHECK_THAT(a.chunk_size == 64, GDN_ERR_UNSUPPORTED, "chunk_size must be 64 (got %d)", a.chunk_size);
  CHECK_THAT(a.T <= MAX_TOKENS && a.V <= (1 << 20), GDN_ERR_UNSUPPORTED,
             "T (%d) must be at most %d and V (%d) at most %d", a.T, MAX_TOKENS, a.V, 1 << 20);
  CHECK_FLAG(a.g_is_cumsum, "g_is_cumsum");
  CHECK_FLAG(a.state_v_first, "state_v_first");
  CHECK_THAT(isfinite(a.scale), GDN_ERR_INVALID_ARG, "scale must be finite");
  if (a.cu_seqlens == nullptr)
    CHECK_THAT(a.N == a.B, GDN_ERR_INVALID_ARG, "without cu_seqlens N (%d) must equal B (%d)", a.N, a.B);
  else
    CHECK_THAT(a.B == 1, GDN_ERR_INVALID_ARG, "with cu_seqlens B must be 1 (got %d)", a.B);
  const int64_t chunks = a.cu_seqlens ? (int64_t)a.N + a.T / 64 : (int64_t)a.B * ((a.T + 63) / 64);
  CHECK_THAT(chunks <= 0x7fffffff, GDN_ERR_UNSUPPORTED, "%lld chunks are too many for one call",
             (long long)chunks);
  if (sizes_only) return GDN_OK;
  if (a.T > 0) {
    CHECK_PTR(a.q, "q");
    CHECK_PTR(a.k, "k");
    CHECK_PTR(a.v, "v");
    CHECK_PTR(a.g, "g");
    CHECK_PTR(a.beta, "beta");
    CHECK_PTR(a.do_, "do");
    CHECK_PTR(a.dq, "dq");
    CHECK_PTR(a.dk, "dk");
    CHECK_PTR(a.dv, "dv");
    CHECK_PTR(a.dg, "dg");
    CHECK_PTR(a.dbeta, "dbeta");
  }
  CHECK_OPT_PTR(a.h0, "h0");
  CHECK_OPT_PTR(a.dht, "dht");
  CHECK_OPT_PTR(a.dh0, "dh0");
  CHECK_OPT_PTR(a.cu_seqlens, "cu_seqlens");
  return GDN_OK;
}

DeltaBwdParams make_params(const gdn_chunk_bwd_args &a) {
  DeltaBwdParams p{};
  p.q = a.q; p.k = a.k; p.v = a.v; p.dout = a.do_; p.g = a.g; p.beta = a.beta; p.h0 = a.h0;
  p.dht = a.dht; p.dq = a.dq; p.dk = a.dk; p.dv = a.dv; p.dg = a.dg; p.dbeta = a.dbeta;
  p.dh0 = a.dh0; p.cu = a.cu_seqlens;
  p.B = a.B; p.T = a.T; p.H = a.H; p.Hg = a.Hg; p.K = a.K; p.V = a.V; p.N = a.N;
  p.g_is_cumsum = a.g_is_cumsum;
  p.v_first = a.state_v_first;
  p.scale = a.scale > 0.f ? a.scale : 1.f / sqrtf((float)a.K);
  p.per_seq = (a.T + 63) / 64;
  p.chunks = a.cu_seqlens ? (int64_t)a.N + a.T / 64 : (int64_t)a.B * p.per_seq;
  p.block = delta_bwd_tc_supported(p, a.dtype == GDN_BF16) ? delta_bwd_tc_block(p)
                                                           : delta_bwd_simt_block(p);
  return p;
}

// The table, rounded up to 256 bytes, then the blocks, then scratch.
size_t table_bytes(const DeltaBwdParams &p) {
  if (p.cu == nullptr) return 0;
  return ((size_t)(2 * (int64_t)p.N + 1 + p.chunks) * sizeof(int32_t) + 255) / 256 * 256;
}

size_t workspace_bytes(const DeltaBwdParams &p, bool bf16) {
  if (p.T == 0) return 0;
  return table_bytes(p) + (size_t)p.chunks * p.H * p.block +
         (delta_bwd_tc_supported(p, bf16) ? delta_bwd_tc_scratch(p) : 0);
}

}  // namespace
}  // namespace gdn

using namespace gdn;

extern "C" {

gdn_status_t gdn_chunk_bwd_workspace_size(const gdn_chunk_bwd_args *a, size_t *bytes) {
  CHECK_THAT(a != nullptr && bytes != nullptr, GDN_ERR_INVALID_ARG, "NULL argument");
  *bytes = 0;
  gdn_status_t st = check_args(*a, true);
  if (st != GDN_OK) return st;
  *bytes = workspace_bytes(make_params(*a), a->dtype == GDN_BF16);
  return GDN_OK;
}

gdn_status_t gdn_chunk_bwd(const gdn_chunk_bwd_args *a, gdn_stream_t stream) {
  (void)set_host_error(GDN_OK, "");
  CHECK_THAT(a != nullptr, GDN_ERR_INVALID_ARG, "args is NULL");
  gdn_status_t st = check_args(*a, false);
  if (st != GDN_OK) return st;
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  DeltaBwdParams p = make_params(*a);
  if (p.T == 0) {
    if (p.dh0 == nullptr && p.cu == nullptr) return GDN_OK;
    p.err = device_error_word();
    if (p.err == nullptr) return launch_status(cudaGetLastError(), "device error word");
    const int64_t values = p.dh0 ? (int64_t)p.N * p.H * p.K * p.V : 0;
    const int64_t blocks = std::min<int64_t>(4 * sm_count(), std::max<int64_t>(1, (values + 255) / 256));
    delta_none_kernel<<<(unsigned)blocks, 256, 0, s>>>(p, values);
    return launch_status(cudaGetLastError(), "state gradient copy");
  }
  const bool bf16 = a->dtype == GDN_BF16;
  const size_t need = workspace_bytes(p, bf16);
  CHECK_THAT(a->workspace != nullptr && a->workspace_bytes >= need, GDN_ERR_WORKSPACE,
             "workspace of %zu bytes needed (got %zu)", need, a->workspace_bytes);
  CHECK_THAT(aligned_to(a->workspace, 256), GDN_ERR_MISALIGNED, "workspace is not 256-byte aligned");
  p.first = static_cast<int32_t *>(a->workspace);
  p.order = p.first + p.N + 1;
  p.owner = p.order + p.N;
  p.blocks = static_cast<unsigned char *>(a->workspace) + table_bytes(p);
  p.scratch = reinterpret_cast<float *>(p.blocks + (size_t)p.chunks * p.H * p.block);
  p.err = device_error_word();
  if (p.err == nullptr) return launch_status(cudaGetLastError(), "device error word");
  if (p.cu != nullptr) {
    delta_table_kernel<<<1, 1024, 0, s>>>(p);
    const cudaError_t e = cudaGetLastError();
    if (e != cudaSuccess) return launch_status(e, "chunk table launch");
  }
  return launch_status(delta_bwd_tc_supported(p, bf16) ? launch_delta_bwd_tc(p, s)
                                                       : launch_delta_bwd_simt(p, bf16, s),
                       "chunk gradient launch");
}

}  // extern "C"
