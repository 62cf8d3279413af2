// Attention over the paged key-value cache, one warp per (query row, head).
//
// For a query at position p of its sequence and the cached keys k_j and
// values v_j, j = 0..p: o = sum_j e^(scale q.k_j - m) v_j / l with the running
// maximum m and sum l = sum_j e^(scale q.k_j - m), and the logarithm of the
// softmax's sum, m + log l. A row that sees no key gives zeros and -inf.
#include "common.cuh"
#include "kernels.h"
#include "layer.cuh"

namespace w4a16 {
namespace {

template <bool kB, bool k8>
__device__ __forceinline__ float cached(const void* base, size_t at) {
  if (k8) return __half2float(__ushort_as_half((unsigned short)e4m3x2_to_half2(static_cast<const uint8_t*>(base)[at])));
  return value16<kB>(static_cast<const uint16_t*>(base)[at]);
}

template <bool kB, bool k8, int D>
__global__ void __launch_bounds__(128) attn_rows_kernel(const AttnArgs a) {
  allow_dependent_launch();
  grid_dependency_wait();
  const int lane = threadIdx.x & 31;
  const long long item = (long long)blockIdx.x * 4 + (threadIdx.x >> 5);
  if (item >= (long long)a.rows * a.heads) return;
  const int row = (int)(item / a.heads), h = (int)(item % a.heads);
  // the row's sequence and how many keys it sees
  int b = row, n = 0;
  if (a.starts) {
    if (row < a.starts[0] || row >= a.starts[a.batch]) return;
    b = 0;
    while (row >= a.starts[b + 1]) ++b;
    n = seq_length(a, b) - (a.starts[b + 1] - 1 - row);
  } else {
    n = seq_length(a, b);
  }
  const int hk = h / (a.heads / a.cache.kv_heads);
  const int page_size = 1 << a.cache.page_shift;
  const float ks = a.cache.k_scale ? a.cache.k_scale[hk] : 1.f, vs = a.cache.v_scale ? a.cache.v_scale[hk] : 1.f;
  float q[D / 32], o[D / 32];
#pragma unroll
  for (int i = 0; i < D / 32; ++i) {
    q[i] = value16<kB>(a.q[(size_t)row * a.ldq + (size_t)h * D + lane + 32 * i]) * a.scale * ks;
    o[i] = 0.f;
  }
  float m = -INFINITY, l = 0.f;
  for (int j = 0; j < n; ++j) {
    const int page = page_of(a, b, j >> a.cache.page_shift);
    const size_t at = (((size_t)page * a.cache.kv_heads + hk) * page_size + (j & (page_size - 1))) * D + lane;
    float s = 0.f;
#pragma unroll
    for (int i = 0; i < D / 32; ++i) s = fmaf(q[i], cached<kB, k8>(a.cache.k, at + 32 * i), s);
#pragma unroll
    for (int w = 16; w > 0; w >>= 1) s += __shfl_xor_sync(0xffffffffu, s, w);
    const float top = fmaxf(m, s);
    const float old = top == -INFINITY ? 1.f : __expf(m - top), p = top == -INFINITY ? 0.f : __expf(s - top);
    m = top;
    l = l * old + p;
#pragma unroll
    for (int i = 0; i < D / 32; ++i) o[i] = o[i] * old + p * cached<kB, k8>(a.cache.v, at + 32 * i);
  }
  const float inv = l > 0.f ? vs / l : 0.f;
#pragma unroll
  for (int i = 0; i < D / 32; ++i) a.out[((size_t)row * a.heads + h) * D + lane + 32 * i] = bits16<kB>(o[i] * inv);
  if (a.lse && lane == 0) a.lse[(size_t)row * a.heads + h] = l > 0.f ? m + __logf(l) : -INFINITY;
}

template <bool kB, bool k8>
cudaError_t launch_rows(const AttnArgs& a, int D, cudaStream_t stream) {
  const dim3 grid((unsigned)(((long long)a.rows * a.heads + 3) / 4));
  return D == 64 ? launch_pdl(attn_rows_kernel<kB, k8, 64>, grid, dim3(128), 0, stream, a)
                 : launch_pdl(attn_rows_kernel<kB, k8, 128>, grid, dim3(128), 0, stream, a);
}

}  // namespace

cudaError_t launch_attn_rows(const AttnArgs& args, int head_dim, bool bf16, bool e4m3, cudaStream_t stream) {
  AttnArgs a = args;
  if (a.rows == 0) return cudaSuccess;
  cudaError_t e = device_error_word(&a.err);
  if (e != cudaSuccess) return e;
  if (bf16) return e4m3 ? launch_rows<true, true>(a, head_dim, stream) : launch_rows<true, false>(a, head_dim, stream);
  return e4m3 ? launch_rows<false, true>(a, head_dim, stream) : launch_rows<false, false>(a, head_dim, stream);
}

}  // namespace w4a16
