// Helpers shared by the kernels of a decoder layer's other operators (norm,
// rotation and cache append, attention): 16-bit and e4m3 conversions, the
// paged cache's addressing, and the launch with programmatic stream
// serialization.
#pragma once

#include <cuda_fp8.h>

#include "common.cuh"
#include "tc_ptx.cuh"

namespace w4a16 {

using tc::allow_dependent_launch;
using tc::grid_dependency_wait;

// Launch with programmatic stream serialization: the grid may be scheduled
// while the previous one drains and waits for it (grid_dependency_wait)
// before it touches memory.
template <class... P, class... A>
cudaError_t launch_pdl(void (*kernel)(P...), dim3 grid, dim3 block, size_t smem, cudaStream_t stream,
                       A&&... args) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = block;
  cfg.dynamicSmemBytes = smem;
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kernel, static_cast<P>(args)...);
}

// 16-bit floats (bf16 with kB, else fp16) from and to fp32.
template <bool kB>
__device__ __forceinline__ float value16(uint32_t bits) {
  return kB ? __uint_as_float(bits << 16) : __half2float(__ushort_as_half((unsigned short)bits));
}
template <bool kB>
__device__ __forceinline__ float2 unpack16(uint32_t v) {
  if (kB) return make_float2(__uint_as_float(v << 16), __uint_as_float(v & 0xffff0000u));
  return __half22float2(*reinterpret_cast<const __half2*>(&v));
}
template <bool kB>
__device__ __forceinline__ uint16_t bits16(float v) {
  return kB ? __bfloat16_as_ushort(__float2bfloat16_rn(v)) : __half_as_ushort(__float2half_rn(v));
}
template <bool kB>
__device__ __forceinline__ uint32_t pack16(float lo, float hi) {
  if (kB) {
    const __nv_bfloat162 b = __floats2bfloat162_rn(lo, hi);
    return *reinterpret_cast<const uint32_t*>(&b);
  }
  const __half2 h = __floats2half2_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&h);
}

// Two e4m3 codes: from fp32 (nearest even, saturating to +-448; NaN stays
// NaN), and to fp16 (exact).
__device__ __forceinline__ uint32_t e4m3x2(float lo, float hi) {
  return __nv_cvt_float2_to_fp8x2(make_float2(lo, hi), __NV_SATFINITE, __NV_E4M3);
}
// Four at a time to two pairs (codes 0, 1 and 2, 3): one instruction each,
// with no code moved to a register of its own.
__device__ __forceinline__ void e4m3x4_to_half2x2(uint32_t codes, uint32_t& lo, uint32_t& hi) {
  asm("{\n\t.reg .b16 l, h;\n\tmov.b32 {l, h}, %2;\n\t"
      "cvt.rn.f16x2.e4m3x2 %0, l;\n\tcvt.rn.f16x2.e4m3x2 %1, h;\n\t}"
      : "=r"(lo), "=r"(hi)
      : "r"(codes));
}

// Elements from the first row's first to the last row's last (for the checked
// build's tests of strided arrays).
__host__ __device__ __forceinline__ size_t span(long long rows, long long stride, long long cols) {
  return rows > 0 ? (size_t)((rows - 1) * stride + cols) : 0;
}

// Error bit of data read on the device that names something outside its
// buffer: a slot, a position, a page number, a length.
constexpr int kErrRange = 128;
// Error bit of a workspace whose flag area was not as every call leaves it.
constexpr int kErrWorkspace = 256;

// The flag area that every workspace starts with; scratch lies behind it.
constexpr size_t kWorkspaceFlags = 32768;

// The paged key-value cache: k and v are [pages][kv heads][page_size][head
// dim] of 16-bit values or of e4m3 codes that a per-head scale multiplies.
struct PagedCache {
  const void* k;
  const void* v;
  const float* k_scale;  // null: 1
  const float* v_scale;
  int pages, page_shift, kv_heads;  // page_size = 1 << page_shift
};

// The arguments of the attention kernels. Rows are query tokens; decode has
// one per sequence (starts null), a prompt's sequence b has the rows
// starts[b] .. starts[b + 1).
struct AttnArgs {
  const uint16_t* q;  // row stride ldq, heads adjacent
  long long ldq;
  PagedCache cache;
  const int32_t* table;  // [batch][max_pages], row stride table_ld
  long long table_ld;
  int max_pages;
  const int32_t* starts;
  const int32_t* lens;
  int rows, batch, heads;
  float scale;
  uint16_t* out;
  float* lse;  // or null
  int* err;
};

// Rows of the cache: [pages][kv heads][page_size].
__device__ __forceinline__ size_t cache_rows(const PagedCache& c) {
  return ((size_t)c.pages * c.kv_heads) << c.page_shift;
}

// A value read on the device that has to lie in [0, most]; one that does not
// is recorded and clamped.
__device__ __forceinline__ int checked(const AttnArgs& a, int v, int most) {
  if (v >= 0 && v <= most) return v;
  atomicOr(a.err, kErrRange);
  return v < 0 ? 0 : most;
}

// What scores are multiplied by before the exponential, as a positive normal
// number: with zero (tiny scales of e4m3 keys, zero queries) a masked score of
// -inf would become NaN. Products of scores with one this small are as good
// as zero.
__device__ __forceinline__ float positive(float mult) { return mult < 1.17549435e-38f ? 1.17549435e-38f : mult; }

// Cached tokens of sequence b, within the capacity of its table row.
__device__ __forceinline__ int seq_length(const AttnArgs& a, int b) {
  return checked(a, *ld_at(a.lens + b, a.lens, (size_t)a.batch, a.err), (int)min((long long)a.max_pages << a.cache.page_shift, 0x7fffffffll));
}

// Page number i of sequence b; one outside the cache is recorded and page 0
// read in its place.
__device__ __forceinline__ int page_of(const AttnArgs& a, int b, int i) {
  const int p = *ld_at(a.table + b * a.table_ld + i, a.table, span(a.batch, a.table_ld, a.max_pages), a.err);
  if ((unsigned)p < (unsigned)a.cache.pages) return p;
  atomicOr(a.err, kErrRange);
  return 0;
}

}  // namespace w4a16
