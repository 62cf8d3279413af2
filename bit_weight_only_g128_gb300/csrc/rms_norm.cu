// Root-mean-square norm with the residual's addition, its result in 16 bits
// or as the 8-bit codes that the W4A8 product takes.
//
// Per row m of K channels, in fp32:
//   h = x + residual,   y = h * (mean_k h^2 + eps)^(-1/2) * weight.
// The residual stream goes on as RNE_16(h) (the one rounding it takes per
// layer), while y is formed from the unrounded h and rounded once. In 8 bits:
// s_a = max_k |y| / 127 (1 for a row of zeros) and the codes
// clamp(round(y / s_a), -127, 127) are taken from the fp32 y, the rule of
// w4a16_quantize_act without its input's rounding to 16 bits.
//
// Bound: HBM bytes, 2 K (x) + 2 K (residual) + 2 K (h) + 2 K or K (y) per
// row; for few rows the chain load - block sum - store (latency). One pass: a
// row's h stays in its threads' registers (at most 4 vectors of 8 channels
// each) from the load to the store. Measured, back to back: 4096 x 8192 bf16 with
// residual 41.6 us, 6450 GB/s (96% of the copy rate); 1 x 4096 1.7 us on the
// device, 4.3 a call; 333 x 5120 to codes 4.2 us on the device, 6 a call.
#include "common.cuh"
#include "kernels.h"
#include "layer.cuh"

namespace w4a16 {
namespace {

struct NormArgs {
  const uint16_t* x;
  const uint16_t* residual;
  const uint16_t* weight;
  uint16_t* y;      // 16-bit result, or null
  uint16_t* codes;  // codes as 16-bit integer values, or null
  int8_t* aq;       // codes as int8, or null
  float* s_a;       // row scales (with codes or aq)
  uint16_t* h;      // residual stream, or null
  long long ldx, ldr, ldh;
  int M, K;
  float eps;
  int* err;
};

// Sum or maximum over the `threads` threads (a multiple of 32) of one row;
// `part` holds one float per warp of the block. Every thread of the block
// takes part.
template <bool kMax>
__device__ __forceinline__ float row_reduce(float v, int warps, float* part) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) {
    const float u = __shfl_xor_sync(0xffffffffu, v, o);
    v = kMax ? fmaxf(v, u) : v + u;
  }
  if (warps == 1) return v;
  const int warp = threadIdx.x >> 5, first = warp / warps * warps;
  if ((threadIdx.x & 31) == 0) part[warp] = v;
  __syncthreads();
  // up to 32 partials: each lane takes one, the same tree in every warp
  const int lane = threadIdx.x & 31;
  v = lane < warps ? part[first + lane] : 0.f;  // (maxima are of magnitudes)
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) {
    const float u = __shfl_xor_sync(0xffffffffu, v, o);
    v = kMax ? fmaxf(v, u) : v + u;
  }
  return v;
}

// kVecs vectors of 8 channels per thread, `row_threads` threads per row, as
// many rows per block as its threads make up.
template <bool kB, int kVecs>
__global__ void __launch_bounds__(1024) rms_norm_kernel(const NormArgs a, int row_threads) {
  __shared__ float part[32], part2[32];
  allow_dependent_launch();
  grid_dependency_wait();
  const int t = threadIdx.x % row_threads;
  const long long m = (long long)blockIdx.x * (blockDim.x / row_threads) + threadIdx.x / row_threads;
  const bool live = m < a.M;
  const int nv = a.K / 8;
  const uint4* xr = reinterpret_cast<const uint4*>(a.x + (live ? m : 0) * a.ldx);
  const uint4* rr = a.residual ? reinterpret_cast<const uint4*>(a.residual + (live ? m : 0) * a.ldr) : nullptr;
  const uint4* wr = reinterpret_cast<const uint4*>(a.weight);
  uint4 xv[kVecs], rv[kVecs], wv[kVecs];
  float h[kVecs][8];
#pragma unroll
  for (int i = 0; i < kVecs; ++i) {
    const int c = t + i * row_threads;
    xv[i] = rv[i] = wv[i] = make_uint4(0, 0, 0, 0);
    if (live && c < nv) {
      xv[i] = ldg_stream(ld_at(xr + c, reinterpret_cast<const uint4*>(a.x), span(a.M, a.ldx, a.K) / 8, a.err));
      if (rr) rv[i] = *ld_at(rr + c, reinterpret_cast<const uint4*>(a.residual), span(a.M, a.ldr, a.K) / 8, a.err);
      if (kVecs <= 2) wv[i] = *ld_at(wr + c, wr, (size_t)nv, a.err);  // in flight with the row (more would not fit the registers)
    }
  }
  float sum = 0.f;
#pragma unroll
  for (int i = 0; i < kVecs; ++i) {
    const uint32_t xw[4] = {xv[i].x, xv[i].y, xv[i].z, xv[i].w};
    const uint32_t rw[4] = {rv[i].x, rv[i].y, rv[i].z, rv[i].w};
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const float2 u = unpack16<kB>(xw[j]), r = unpack16<kB>(rw[j]);
      h[i][2 * j] = u.x + r.x;
      h[i][2 * j + 1] = u.y + r.y;
      sum = fmaf(h[i][2 * j], h[i][2 * j], sum);
      sum = fmaf(h[i][2 * j + 1], h[i][2 * j + 1], sum);
    }
  }
  const int warps = row_threads / 32;
  sum = row_reduce<false>(sum, warps, part);
  const float scale = rsqrtf(sum / (float)a.K + a.eps);
  float top = 0.f;
#pragma unroll
  for (int i = 0; i < kVecs; ++i) {
    const int c = t + i * row_threads;
    if (live && c < nv) {
      if (a.h) {
        uint4 o;
        o.x = pack16<kB>(h[i][0], h[i][1]);
        o.y = pack16<kB>(h[i][2], h[i][3]);
        o.z = pack16<kB>(h[i][4], h[i][5]);
        o.w = pack16<kB>(h[i][6], h[i][7]);
        uint4* d = reinterpret_cast<uint4*>(a.h + m * a.ldh) + c;
        if (in_buf(d, reinterpret_cast<uint4*>(a.h), span(a.M, a.ldh, a.K) / 8, a.err)) *d = o;
      }
      const uint4 w = kVecs <= 2 ? wv[i] : *ld_at(wr + c, wr, (size_t)nv, a.err);
      const uint32_t ww[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const float2 g = unpack16<kB>(ww[j]);
        h[i][2 * j] = h[i][2 * j] * scale * g.x;
        h[i][2 * j + 1] = h[i][2 * j + 1] * scale * g.y;
        top = fmaxf(top, fmaxf(fabsf(h[i][2 * j]), fabsf(h[i][2 * j + 1])));
      }
      if (a.y) {
        uint4 o;
        o.x = pack16<kB>(h[i][0], h[i][1]);
        o.y = pack16<kB>(h[i][2], h[i][3]);
        o.z = pack16<kB>(h[i][4], h[i][5]);
        o.w = pack16<kB>(h[i][6], h[i][7]);
        uint4* d = reinterpret_cast<uint4*>(a.y + m * a.K) + c;
        if (in_buf(d, reinterpret_cast<uint4*>(a.y), (size_t)a.M * nv, a.err)) *d = o;
      }
    }
  }
  if (!a.s_a) return;
  top = row_reduce<true>(top, warps, part2);
  if (!live) return;
  const float s = act_scale(top);
  const float inv = __frcp_rn(s);
  if (t == 0 && in_buf(a.s_a + m, a.s_a, (size_t)a.M, a.err)) a.s_a[m] = s;
#pragma unroll
  for (int i = 0; i < kVecs; ++i) {
    const int c = t + i * row_threads;
    if (c >= nv) break;
#pragma unroll
    for (int j = 0; j < 8; ++j) h[i][j] = act_code(h[i][j], s, inv);
    if (a.codes) {
      uint4 o;
      o.x = pack16<kB>(h[i][0], h[i][1]);
      o.y = pack16<kB>(h[i][2], h[i][3]);
      o.z = pack16<kB>(h[i][4], h[i][5]);
      o.w = pack16<kB>(h[i][6], h[i][7]);
      uint4* d = reinterpret_cast<uint4*>(a.codes + m * a.K) + c;
      if (in_buf(d, reinterpret_cast<uint4*>(a.codes), (size_t)a.M * nv, a.err)) *d = o;
    }
    if (a.aq) {
      uint32_t lo = 0, hi = 0;
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        lo |= ((uint32_t)(int)h[i][j] & 0xffu) << (8 * j);
        hi |= ((uint32_t)(int)h[i][4 + j] & 0xffu) << (8 * j);
      }
      uint2* d = reinterpret_cast<uint2*>(a.aq + m * a.K) + c;
      if (in_buf(d, reinterpret_cast<uint2*>(a.aq), (size_t)a.M * nv, a.err)) *d = make_uint2(lo, hi);
    }
  }
}

// Any K (above 32768 a row does not fit the registers), stride and 2-byte
// alignment: one block per row, the row read again
// for each of the steps (sum, maximum, result). An output that is the
// residual itself is written in the last step only, each element by the
// thread that reads it.
template <bool kB>
__global__ void __launch_bounds__(256) rms_norm_any_kernel(const NormArgs a) {
  __shared__ float part[32], part2[32];
  allow_dependent_launch();
  grid_dependency_wait();
  const long long m = blockIdx.x;
  const uint16_t* xr = a.x + m * a.ldx;
  const uint16_t* rr = a.residual ? a.residual + m * a.ldr : nullptr;
  auto value = [&](int k) {
    return value16<kB>(*ld_at(xr + k, a.x, span(a.M, a.ldx, a.K), a.err)) +
           (rr ? value16<kB>(*ld_at(rr + k, a.residual, span(a.M, a.ldr, a.K), a.err)) : 0.f);
  };
  auto weight = [&](int k) { return value16<kB>(*ld_at(a.weight + k, a.weight, (size_t)a.K, a.err)); };
  auto store = [&](auto* base, long long ld, int k, auto v) {
    auto* d = base + m * ld + k;
    if (in_buf(d, base, span(a.M, ld, a.K), a.err)) *d = v;
  };
  float sum = 0.f;
  for (int k = threadIdx.x; k < a.K; k += 256) {
    const float v = value(k);
    sum = fmaf(v, v, sum);
  }
  sum = row_reduce<false>(sum, 8, part);
  const float scale = rsqrtf(sum / (float)a.K + a.eps);
  float s = 1.f, inv = 1.f;
  if (a.s_a) {
    float top = 0.f;
    for (int k = threadIdx.x; k < a.K; k += 256)
      top = fmaxf(top, fabsf(value(k) * scale * weight(k)));
    top = row_reduce<true>(top, 8, part2);
    s = act_scale(top);
    inv = __frcp_rn(s);
    if (threadIdx.x == 0) store(a.s_a, 1, 0, s);
  }
  for (int k = threadIdx.x; k < a.K; k += 256) {
    const float v = value(k);
    const float y = v * scale * weight(k);
    if (a.h) store(a.h, a.ldh, k, bits16<kB>(v));
    if (a.y) store(a.y, a.K, k, bits16<kB>(y));
    if (a.s_a) {
      const float c = act_code(y, s, inv);
      if (a.codes) store(a.codes, a.K, k, bits16<kB>(c));
      if (a.aq) store(a.aq, a.K, k, (int8_t)(int)c);
    }
  }
}

template <bool kB>
cudaError_t launch_norm(const NormArgs& a, cudaStream_t stream) {
  auto al = [](const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15) == 0; };
  const bool vec = a.K % 8 == 0 && a.K <= 32768 && a.ldx % 8 == 0 && a.ldr % 8 == 0 && a.ldh % 8 == 0 && al(a.x) &&
                   al(a.residual) && al(a.weight) && al(a.y) && al(a.codes) && al(a.aq) && al(a.h);
  if (!vec) return launch_pdl(rms_norm_any_kernel<kB>, dim3((unsigned)a.M), dim3(256), 0, stream, a);
  const int nv = a.K / 8;
  // Vectors per thread: one in short rows; two while all rows' threads fit the
  // device at once (then a row's chain of loads, sums and stores is what
  // counts, and fewer warps join sooner: 333 x 5120 codes 4.4 us with two, 5.2
  // with one, 6.1 with four); four beyond that (bytes in flight of the resident
  // blocks: 4096 x 8192 41.6 us with four, 47.7 with two, 50.9 with one).
  int vecs = nv <= 128 ? 1 : nv <= 2048 ? 2 : 4;
  while (vecs < 4 && (long long)a.M * ((nv + vecs - 1) / vecs) > (long long)device_sms() * 2048) vecs *= 2;
  int threads = ((nv + vecs - 1) / vecs + 31) / 32 * 32;
  int rows = threads >= 128 ? 1 : 128 / threads;
  if (rows > a.M) rows = a.M;
  const dim3 grid((unsigned)((a.M + rows - 1) / rows)), block((unsigned)(rows * threads));
  switch (vecs) {
    case 1: return launch_pdl(rms_norm_kernel<kB, 1>, grid, block, 0, stream, a, threads);
    case 2: return launch_pdl(rms_norm_kernel<kB, 2>, grid, block, 0, stream, a, threads);
    default: return launch_pdl(rms_norm_kernel<kB, 4>, grid, block, 0, stream, a, threads);
  }
}

}  // namespace

cudaError_t launch_rms_norm(const uint16_t* x, long long ldx, const uint16_t* residual, long long ldr,
                            const uint16_t* weight, int M, int K, float eps, bool bf16, uint16_t* y,
                            uint16_t* codes, int8_t* aq, float* s_a, uint16_t* h, long long ldh,
                            cudaStream_t stream) {
  if (M == 0) return cudaSuccess;
  NormArgs a = {x, residual, weight, y, codes, aq, s_a, h, ldx, ldr, ldh, M, K, eps, nullptr};
  cudaError_t e = device_error_word(&a.err);
  if (e != cudaSuccess) return e;
  return bf16 ? launch_norm<true>(a, stream) : launch_norm<false>(a, stream);
}

}  // namespace w4a16
