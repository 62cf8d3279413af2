// Rotation of queries and keys by their positions, with the keys and values
// appended to the paged cache on the way.
//
// Per token t at position p, for the first R dimensions of every query and
// key head, with (c_i, s_i) = (cos, sin) row p of the table, i < R/2:
//   (a, b) -> (a c_i - b s_i, b c_i + a s_i)
// where (a, b) are the dimensions (i, i + R/2), or (2i, 2i + 1) interleaved;
// the other dimensions and the values pass through. Products and sums are
// fp32; each result is rounded once, to 16 bits, or to the cache's e4m3 codes
// of x times the fp32 reciprocal of scale[head].
//
// Bound: HBM bytes (the qkv rows in, q and the cache rows out); for a few
// tokens the chain slot/position - table row - store (latency). Each thread
// takes both halves of a rotated pair as two 16-byte vectors, for two heads.
// Measured, back to back: 4001 tokens of 64 heads over 8 into e4m3 27.1 us a
// call, 5830 GB/s (25.2 on the device); 16 tokens of 32 heads 1.8 us on the
// device, 3.9 a call.
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
__global__ void __launch_bounds__(kMostThreads, 2) rope_append_kernel(const RopeArgs a) {
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
  uint4 x[2][2] = {};
#pragma unroll
  for (int n = 0; n < 2; ++n) {
    const int h = h0 + n * stride;
    if (h < heads) {
      const size_t all = span(a.T, a.ld, heads * D) - 7;
      x[n][0] = ldg_now(ld_at(row + (size_t)h * D + d0, a.qkv, all, a.err));
      x[n][1] = ldg_now(ld_at(row + (size_t)h * D + d1, a.qkv, all, a.err));
    }
  }
  const long long slot = *ld_at(a.slots + t, a.slots, (size_t)a.T, a.err);
  int pos = *ld_at(a.positions + t, a.positions, (size_t)a.T, a.err);
  bool keep = slot >= 0;
  if (slot >= a.capacity || pos < 0 || pos >= a.table_len) {
    if (threadIdx.x == 0) atomicOr(a.err, kErrRange);
    if (slot >= a.capacity) keep = false;
    if (pos < 0 || pos >= a.table_len) pos = 0;
  }
  const int page_size = 1 << a.page_shift;
  const size_t page = keep ? (size_t)(slot >> a.page_shift) : 0;
  const int off = keep ? (int)(slot & (page_size - 1)) : 0;
  const float* cosines = a.table + (size_t)pos * a.R + 8 * j;
  if (turned) cosines = ld_at(cosines, a.table, (size_t)a.table_len * a.R - half - 7, a.err);
  const float* sines = cosines + half;
  float inv[2];  // of the head's e4m3 scale
#pragma unroll
  for (int n = 0; n < 2; ++n) {
    const int h = h0 + n * stride;
    inv[n] = 1.f;
    if (k8 && h >= a.heads && h < heads)
      inv[n] = __frcp_rn(h < a.heads + a.kv_heads
                             ? *ld_at(a.k_scale + h - a.heads, a.k_scale, (size_t)a.kv_heads, a.err)
                             : *ld_at(a.v_scale + h - a.heads - a.kv_heads, a.v_scale, (size_t)a.kv_heads, a.err));
  }
  // two dimensions of each vector at a time, in place (an e4m3 pair takes the
  // word's lower half)
#pragma unroll
  for (int w = 0; w < 4; ++w) {
    float2 c = make_float2(1.f, 1.f), s = make_float2(0.f, 0.f);
    if (turned) {
      // interleaved: word w of the first vector turns by angle w, of the
      // second by angle 4 + w; else both words by angles 2w and 2w + 1
      c = kInter ? make_float2(cosines[w], cosines[4 + w]) : *reinterpret_cast<const float2*>(cosines + 2 * w);
      s = kInter ? make_float2(sines[w], sines[4 + w]) : *reinterpret_cast<const float2*>(sines + 2 * w);
    }
#pragma unroll
    for (int n = 0; n < 2; ++n) {
      const int h = h0 + n * stride;
      const bool is_q = h < a.heads, is_v = h >= a.heads + a.kv_heads;
      uint32_t& x0 = reinterpret_cast<uint32_t(&)[4]>(x[n][0])[w];
      uint32_t& x1 = reinterpret_cast<uint32_t(&)[4]>(x[n][1])[w];
      float2 lo = unpack16<kB>(x0), hi = unpack16<kB>(x1);
      if (turned && !is_v) {
        const float2 u = lo, v = hi;
        if (kInter) {
          lo = make_float2(u.x * c.x - u.y * s.x, u.y * c.x + u.x * s.x);
          hi = make_float2(v.x * c.y - v.y * s.y, v.y * c.y + v.x * s.y);
        } else {
          lo = make_float2(u.x * c.x - v.x * s.x, u.y * c.y - v.y * s.y);
          hi = make_float2(v.x * c.x + u.x * s.x, v.y * c.y + u.y * s.y);
        }
      }
      if (k8 && !is_q) {
        x0 = e4m3x2(lo.x * inv[n], lo.y * inv[n]);
        x1 = e4m3x2(hi.x * inv[n], hi.y * inv[n]);
      } else {
        x0 = pack16<kB>(lo.x, lo.y);
        x1 = pack16<kB>(hi.x, hi.y);
      }
    }
  }
#pragma unroll
  for (int n = 0; n < 2; ++n) {
    const int h = h0 + n * stride;
    if (h >= heads) break;
    const bool is_q = h < a.heads, is_v = h >= a.heads + a.kv_heads;
    if (is_q) {
      uint16_t* q = a.q + ((size_t)t * a.heads + h) * D;
      const size_t all = (size_t)a.T * a.heads * D - 7;
      if (!in_buf(q + d0, a.q, all, a.err) || !in_buf(q + d1, a.q, all, a.err)) continue;
      *reinterpret_cast<uint4*>(q + d0) = x[n][0];
      *reinterpret_cast<uint4*>(q + d1) = x[n][1];
    } else if (keep) {
      const int hk = is_v ? h - a.heads - a.kv_heads : h - a.heads;
      const size_t at = ((page * a.kv_heads + hk) * page_size + off) * D;
      const size_t all = (size_t)a.capacity * a.kv_heads * D - 7;
      void* base = is_v ? a.v : a.k;
      if (k8) {
        uint8_t* to = static_cast<uint8_t*>(base) + at;
        if (!in_buf(to + d0, static_cast<uint8_t*>(base), all, a.err) || !in_buf(to + d1, static_cast<uint8_t*>(base), all, a.err)) continue;
        *reinterpret_cast<uint2*>(to + d0) = make_uint2(x[n][0].x | (x[n][0].y << 16), x[n][0].z | (x[n][0].w << 16));
        *reinterpret_cast<uint2*>(to + d1) = make_uint2(x[n][1].x | (x[n][1].y << 16), x[n][1].z | (x[n][1].w << 16));
      } else {
        uint16_t* to = static_cast<uint16_t*>(base) + at;
        if (!in_buf(to + d0, static_cast<uint16_t*>(base), all, a.err) || !in_buf(to + d1, static_cast<uint16_t*>(base), all, a.err)) continue;
        *reinterpret_cast<uint4*>(to + d0) = x[n][0];
        *reinterpret_cast<uint4*>(to + d1) = x[n][1];
      }
    }
  }
}

// Any even R, stride and 2-byte alignment of qkv: one thread per element.
template <bool kB, bool k8, bool kInter>
__global__ void __launch_bounds__(kThreads) rope_append_any_kernel(const RopeArgs a, int D) {
  allow_dependent_launch();
  grid_dependency_wait();
  const int t = blockIdx.x;
  const long long slot = *ld_at(a.slots + t, a.slots, (size_t)a.T, a.err);
  int pos = *ld_at(a.positions + t, a.positions, (size_t)a.T, a.err);
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
    auto at16 = [&](int i) { return value16<kB>(*ld_at(x + i, a.qkv, span(a.T, a.ld, heads * D), a.err)); };
    auto angle = [&](int i) { return *ld_at(turn + i, a.table, (size_t)a.table_len * a.R, a.err); };
    float f = at16(d);
    if (d < a.R && !is_v) {
      const bool first = kInter ? d % 2 == 0 : d < half;
      const int k = kInter ? d / 2 : (first ? d : d - half);
      const float g = at16(kInter ? (first ? d + 1 : d - 1) : (first ? d + half : d - half));
      f = first ? f * angle(k) - g * angle(half + k) : f * angle(k) + g * angle(half + k);
    }
    if (is_q) {
      uint16_t* q = a.q + ((size_t)t * a.heads + h) * D + d;
      if (in_buf(q, a.q, (size_t)a.T * a.heads * D, a.err)) *q = bits16<kB>(f);
      continue;
    }
    const int hk = is_v ? h - a.heads - a.kv_heads : h - a.heads;
    const size_t at = ((page * a.kv_heads + hk) * page_size + off) * D + d;
    void* base = is_v ? a.v : a.k;
    if (!in_buf(static_cast<uint8_t*>(base) + at, static_cast<uint8_t*>(base), (size_t)a.capacity * a.kv_heads * D, a.err)) continue;
    if (k8)
      static_cast<uint8_t*>(base)[at] = (uint8_t)e4m3x2(f * __frcp_rn(*ld_at((is_v ? a.v_scale : a.k_scale) + hk, is_v ? a.v_scale : a.k_scale, (size_t)a.kv_heads, a.err)), 0.f);
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
