// What the kernels of the products grouped by expert share (experts.cu:
// few rows per expert; experts_tc.cu: many).
//
// The weights of E experts are one packed weight of E * N columns: expert e's
// strips are e * N/16 .. (e + 1) * N/16, so that no kernel needs a pointer per
// expert. The rows of the products are the choices f = token * top + j of the
// router: `rows` lists them by expert, expert e's at offsets[e] ..
// offsets[e + 1), those of no expert from offsets[E] on. Choice f multiplies
// row f / top of A, or row f where A has a row per choice, and its result is
// row f of the output, whatever its place in `rows`.
#pragma once

#include "common.cuh"
#include "kernels.h"
#include "layer.cuh"

namespace w4a16 {

struct ExpertArgs {
  const uint16_t* A;      // [T or T * top][K]
  const uint32_t* Wq;
  const uint16_t* Sp;
  const uint32_t* Zp;
  const int32_t* experts;  // [T * top]
  const float* weights;    // [T * top], or null
  const int32_t* rows;     // [T * top]
  const int32_t* offsets;  // [E + 1]
  uint16_t* Y;             // [T * top][silu ? N/2 : N]; combined [T][N]
  int T, top, E, N, K, group;
  int per_choice;          // A has a row per choice
  int silu, combine;
  int* err;
};

__host__ __device__ __forceinline__ int choices(const ExpertArgs& a) { return a.T * a.top; }

// offsets[e] as data from outside: within [0, T * top].
__device__ __forceinline__ int offset_of(const ExpertArgs& a, int e) {
  const int v = *ld_at(a.offsets + e, a.offsets, (size_t)a.E + 1, a.err), most = choices(a);
  if (v >= 0 && v <= most) return v;
  atomicOr(a.err, kErrRange);
  return v < 0 ? 0 : most;
}

// Choice number i of `rows`; -1 (recorded) where it names none.
__device__ __forceinline__ int choice_of(const ExpertArgs& a, int i) {
  const int f = *ld_at(a.rows + i, a.rows, (size_t)choices(a), a.err);
  if ((unsigned)f < (unsigned)choices(a)) return f;
  atomicOr(a.err, kErrRange);
  return -1;
}

__device__ __forceinline__ size_t a_elements(const ExpertArgs& a) {
  return (size_t)(a.per_choice ? choices(a) : a.T) * a.K;
}

// Asynchronous copies of 16 and 4 bytes to shared memory.
__device__ __forceinline__ void copy16(uint32_t to, const void* from) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(to), "l"(from) : "memory");
}
__device__ __forceinline__ void copy4(uint32_t to, const void* from) {
  asm volatile("cp.async.ca.shared.global [%0], [%1], 4;" ::"r"(to), "l"(from) : "memory");
}

// silu(g) * u in fp32.
__device__ __forceinline__ float silu_times(float g, float u) { return __fdividef(g, 1.f + __expf(-g)) * u; }

}  // namespace w4a16
