// Rotation of queries and keys by their positions, with the keys and values
// appended to the paged cache on the way.
//
// Per token t at position p, for the first R dimensions of every query and
// key head, with (c_i, s_i) = (cos, sin) row p of the table, i < R/2:
//   (a, b) -> (a c_i - b s_i, b c_i + a s_i)
// where (a, b) are the dimensions (i, i + R/2), or (2i, 2i + 1) interleaved;
// the other dimensions and the values pass through. Products and sums are
// fp32; each result is rounded once, to 16 bits or to the cache's e4m3 codes
// of x / scale[head].
//
// Bound: HBM bytes (the qkv rows in, q and the cache rows out); for a few
// tokens the chain slot/position - table row - store (latency). Each thread
// takes both halves of a rotated pair as two 16-byte vectors and keeps its
// cosines and sines in registers over the heads that it takes.
#include "common.cuh"
#include "kernels.h"
#include "layer.cuh"

namespace w4a16 {
namespace {

struct RopeArgs {
  const uint16_t* qkv;
  const float* table;  // [table_len][R]: cosines, then sines
  const int32_t* positions;
  const int64_t* slots;
  uint16_t* q;
  void* k;
  void* v;
  const float* k_scale;
  const float* v_scale;
  long long ld;  // row stride of qkv
  long long capacity;  // pages * page_size
  int table_len, R, T, heads, kv_heads, page_shift;
  int* err;
};

template <bool kB>
__device__ __forceinline__ uint4 pack8(const float (&f)[8]) {
  return make_uint4(pack16<kB>(f[0], f[1]), pack16<kB>(f[2], f[3]), pack16<kB>(f[4], f[5]), pack16<kB>(f[6], f[7]));
}
template <bool kB>
__device__ __forceinline__ void unpack8(const uint4& v, float (&f)[8]) {
  const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float2 u = unpack16<kB>(w[i]);
    f[2 * i] = u.x;
    f[2 * i + 1] = u.y;
  }
}

// 8 consecutive values to q or the cache, at element `at` (e4m3: f * inv).
template <bool kB, bool k8>
__device__ __forceinline__ void store8(void* base, size_t at, const float (&f)[8], float inv) {
  if (k8) {
    float g[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) g[i] = f[i] * inv;
    uint2 o;
    o.x = e4m3x2(g[0], g[1]) | (e4m3x2(g[2], g[3]) << 16);
    o.y = e4m3x2(g[4], g[5]) | (e4m3x2(g[6], g[7]) << 16);
    *reinterpret_cast<uint2*>(static_cast<uint8_t*>(base) + at) = o;
  } else {
    *reinterpret_cast<uint4*>(static_cast<uint16_t*>(base) + at) = pack8<kB>(f);
  }
}

constexpr int kThreads = 256;    // of the element path
constexpr int kMostThreads = 512;  // of the vector path

// A load that stays where it is written: ahead of the loads that the block
// waits for.
__device__ __forceinline__ uint4 ldg_now(const uint16_t* p) {
  uint4 v;
  asm volatile("ld.global.nc.L1::no_allocate.v4.u32 {%0, %1, %2, %3}, [%4];"
               : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
               : "l"(p));
  return v;
}

// R a multiple of 16. D / 16 threads per head, each with two vectors of 8:
// the halves of a pair below R, consecutive ones above. A thread takes two
// heads, whose four vectors are in flight while the slot, the position and
// the table's row arrive. blockIdx.x: token, blockIdx.y: share of the heads.
template <bool kB, bool k8, bool kInter, int D>
__global__ void __launch_bounds__(kMostThreads) rope_append_kernel(const RopeArgs a) {
  constexpr int kLanes = D / 16;  // threads per head
  allow_dependent_launch();
  grid_dependency_wait();
  const int t = blockIdx.x;
  const int j = threadIdx.x % kLanes;
  const int heads = a.heads + 2 * a.kv_heads, stride = blockDim.x / kLanes;
  const bool turned = 16 * j < a.R;
  const int half = a.R / 2;
  // the two vectors' first dimensions
  const int d0 = turned && !kInter ? 8 * j : 16 * j;
  const int d1 = turned && !kInter ? half + 8 * j : 16 * j + 8;
  const uint16_t* row = a.qkv + (size_t)t * a.ld;
  const int h0 = blockIdx.y * 2 * stride + threadIdx.x / kLanes;
  uint4 x[2][2];
#pragma unroll
  for (int n = 0; n < 2; ++n) {
    const int h = h0 + n * stride;
    if (h < heads) {
      x[n][0] = ldg_now(row + (size_t)h * D + d0);
      x[n][1] = ldg_now(row + (size_t)h * D + d1);
    }
  }
  const long long slot = a.slots[t];
  int pos = a.positions[t];
  bool keep = slot >= 0;
  if (slot >= a.capacity || pos < 0 || pos >= a.table_len) {
    if (threadIdx.x == 0) atomicOr(a.err, kErrRange);
    if (slot >= a.capacity) keep = false;
    if (pos < 0 || pos >= a.table_len) pos = 0;
  }
  float c[8], s[8];
  if (turned) {
    const float4* angles = reinterpret_cast<const float4*>(a.table + (size_t)pos * a.R);
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const float4 u = angles[2 * j + i], w = angles[half / 4 + 2 * j + i];
      c[4 * i] = u.x, c[4 * i + 1] = u.y, c[4 * i + 2] = u.z, c[4 * i + 3] = u.w;
      s[4 * i] = w.x, s[4 * i + 1] = w.y, s[4 * i + 2] = w.z, s[4 * i + 3] = w.w;
    }
  }
  const int page_size = 1 << a.page_shift;
  const size_t page = keep ? (size_t)(slot >> a.page_shift) : 0;
  const int off = keep ? (int)(slot & (page_size - 1)) : 0;
#pragma unroll
  for (int n = 0; n < 2; ++n) {
    const int h = h0 + n * stride;
    if (h >= heads) break;
    const bool is_q = h < a.heads, is_v = h >= a.heads + a.kv_heads;
    if (!is_q && !keep) continue;
    float lo[8], hi[8];
    unpack8<kB>(x[n][0], lo);
    unpack8<kB>(x[n][1], hi);
    if (turned && !is_v) {
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        if (kInter) {
          // 16 consecutive dimensions: pairs (0,1) .. (6,7) of lo, then of hi
          float& u0 = i < 4 ? lo[2 * i] : hi[2 * i - 8];
          float& w0 = i < 4 ? lo[2 * i + 1] : hi[2 * i - 7];
          const float u = u0 * c[i] - w0 * s[i], w = w0 * c[i] + u0 * s[i];
          u0 = u, w0 = w;
        } else {
          const float u = lo[i] * c[i] - hi[i] * s[i], w = hi[i] * c[i] + lo[i] * s[i];
          lo[i] = u, hi[i] = w;
        }
      }
    }
    if (is_q) {
      const size_t at = ((size_t)t * a.heads + h) * D;
      store8<kB, false>(a.q, at + d0, lo, 1.f);
      store8<kB, false>(a.q, at + d1, hi, 1.f);
    } else {
      const int hk = is_v ? h - a.heads - a.kv_heads : h - a.heads;
      const size_t at = ((page * a.kv_heads + hk) * page_size + off) * D;
      const float inv = k8 ? __frcp_rn((is_v ? a.v_scale : a.k_scale)[hk]) : 1.f;
      store8<kB, k8>(is_v ? a.v : a.k, at + d0, lo, inv);
      store8<kB, k8>(is_v ? a.v : a.k, at + d1, hi, inv);
    }
  }
}

// Any even R, stride and 2-byte alignment of qkv: one thread per element.
template <bool kB, bool k8, bool kInter>
__global__ void __launch_bounds__(kThreads) rope_append_any_kernel(const RopeArgs a, int D) {
  allow_dependent_launch();
  grid_dependency_wait();
  const int t = blockIdx.x;
  const long long slot = a.slots[t];
  int pos = a.positions[t];
  bool keep = slot >= 0;
  if (slot >= a.capacity || pos < 0 || pos >= a.table_len) {
    if (threadIdx.x == 0) atomicOr(a.err, kErrRange);
    if (slot >= a.capacity) keep = false;
    if (pos < 0 || pos >= a.table_len) pos = 0;
  }
  const int half = a.R / 2, heads = a.heads + 2 * a.kv_heads, page_size = 1 << a.page_shift;
  const float* turn = a.table + (size_t)pos * a.R;
  const size_t page = keep ? (size_t)(slot >> a.page_shift) : 0;
  const int off = keep ? (int)(slot & (page_size - 1)) : 0;
  for (int i = blockIdx.y * kThreads + threadIdx.x; i < heads * D; i += gridDim.y * kThreads) {
    const int h = i / D, d = i - h * D;
    const bool is_q = h < a.heads, is_v = h >= a.heads + a.kv_heads;
    if (!is_q && !keep) continue;
    const uint16_t* x = a.qkv + (size_t)t * a.ld + (size_t)h * D;
    float f = value16<kB>(x[d]);
    if (d < a.R && !is_v) {
      const bool first = kInter ? d % 2 == 0 : d < half;
      const int k = kInter ? d / 2 : (first ? d : d - half);
      const float g = value16<kB>(x[kInter ? (first ? d + 1 : d - 1) : (first ? d + half : d - half)]);
      f = first ? f * turn[k] - g * turn[half + k] : f * turn[k] + g * turn[half + k];
    }
    if (is_q) {
      a.q[((size_t)t * a.heads + h) * D + d] = bits16<kB>(f);
      continue;
    }
    const int hk = is_v ? h - a.heads - a.kv_heads : h - a.heads;
    const size_t at = ((page * a.kv_heads + hk) * page_size + off) * D + d;
    void* base = is_v ? a.v : a.k;
    if (k8)
      static_cast<uint8_t*>(base)[at] = (uint8_t)e4m3x2(f * __frcp_rn((is_v ? a.v_scale : a.k_scale)[hk]), 0.f);
    else
      static_cast<uint16_t*>(base)[at] = bits16<kB>(f);
  }
}

template <bool kB, bool k8, bool kInter>
cudaError_t launch_rope(const RopeArgs& a, int D, cudaStream_t stream) {
  const int heads = a.heads + 2 * a.kv_heads;
  auto al = [](const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15) == 0; };
  if (a.R % 16 != 0 || a.ld % 8 != 0 || !al(a.qkv) || !al(a.q) || !al(a.table)) {
    // a token over several blocks while the tokens are few
    const int steps = (heads * D + kThreads - 1) / kThreads, share = (device_sms() * 4 + a.T - 1) / a.T;
    return launch_pdl(rope_append_any_kernel<kB, k8, kInter>, dim3((unsigned)a.T, (unsigned)(share < steps ? share : steps)),
                      dim3(kThreads), 0, stream, a, D);
  }
  // two heads per thread, in as few blocks per token as hold them, evenly
  const int tasks = (heads + 1) / 2 * (D / 16);
  const int blocks = (tasks + kMostThreads - 1) / kMostThreads;
  const int threads = ((tasks + blocks - 1) / blocks + 31) / 32 * 32;
  const dim3 grid((unsigned)a.T, (unsigned)blocks);
  return D == 64 ? launch_pdl(rope_append_kernel<kB, k8, kInter, 64>, grid, dim3(threads), 0, stream, a)
                 : launch_pdl(rope_append_kernel<kB, k8, kInter, 128>, grid, dim3(threads), 0, stream, a);
}

}  // namespace

cudaError_t launch_rope_append(const uint16_t* qkv, long long ld, const float* table, int table_len, int R,
                               const int32_t* positions, const int64_t* slots, int T, int heads, int kv_heads,
                               int head_dim, uint16_t* q, void* k, void* v, const float* k_scale,
                               const float* v_scale, int pages, int page_shift, bool bf16, bool e4m3,
                               bool interleaved, cudaStream_t stream) {
  if (T == 0) return cudaSuccess;
  RopeArgs a = {qkv, table, positions, slots, q, k, v, k_scale, v_scale, ld, (long long)pages << page_shift,
                table_len, R, T, heads, kv_heads, page_shift, nullptr};
  cudaError_t e = device_error_word(&a.err);
  if (e != cudaSuccess) return e;
  switch ((bf16 ? 4 : 0) | (e4m3 ? 2 : 0) | (interleaved ? 1 : 0)) {
    case 0: return launch_rope<false, false, false>(a, head_dim, stream);
    case 1: return launch_rope<false, false, true>(a, head_dim, stream);
    case 2: return launch_rope<false, true, false>(a, head_dim, stream);
    case 3: return launch_rope<false, true, true>(a, head_dim, stream);
    case 4: return launch_rope<true, false, false>(a, head_dim, stream);
    case 5: return launch_rope<true, false, true>(a, head_dim, stream);
    case 6: return launch_rope<true, true, false>(a, head_dim, stream);
    default: return launch_rope<true, true, true>(a, head_dim, stream);
  }
}

}  // namespace w4a16
