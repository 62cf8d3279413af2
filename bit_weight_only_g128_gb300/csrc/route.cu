// The router of a layer of experts: each token's experts and their weights,
// and the choices in the experts' order for the products grouped by expert.
//
// Per token, its experts are the top_k largest logits, in descending order,
// equal ones by the lower index (NaN before everything, -0 equal to +0); a
// logit of -inf is never chosen. With m the largest logit, a chosen one x
// scores exp(x - m) / sum_e exp(x_e - m), or 1 / (1 + exp(-x)); renormalized,
// the scores are divided by their sum instead. The choices f = token * top_k +
// j are then sorted by expert, stably (a counting sort: per-block histograms,
// a prefix over experts and blocks, ranks by matching within a warp), those
// of no expert last. All counts are integers, so the order of the atomics
// changes nothing; exponentials and sums are fp32.
//
// A warp takes a token: its logits lie in registers, the maximum of the
// ordered bit patterns and then the lowest index that has it are one
// reduction instruction each.
//
// Bound: latency. The logits of a prompt are a megabyte or so; what counts is
// the chain of k dependent reductions per token and the launches. Up to
// kOneBlock tokens one block does everything in one launch; above it a second
// kernel places the choices once every block's counts are known.
// Measured (top 8 of 64, a call; in a graph): 1 token 4.7-5.3 us, 3.0; 4099 tokens
// 10-20 us from process to process (the same binary; 19-20 where the inputs
// change from call to call), 9.8 (1.4 MB moved: 0.15 TB/s).
#include "common.cuh"
#include "kernels.h"
#include "layer.cuh"

namespace w4a16 {
namespace {

constexpr int kThreads = 512;
constexpr int kWarps = kThreads / 32;
constexpr int kOneBlock = 64;  // tokens
constexpr int kBlocks = 76;    // most blocks of the two-kernel form
constexpr uint32_t kFull = 0xffffffffu;
constexpr uint32_t kLowest = 0x007fffffu;  // the ordered pattern of -inf

struct RouteArgs {
  const void* logits;
  long long ld;
  int type;  // 0: fp16, 1: bf16, 2: fp32
  int T, E, k, sigmoid, renormalize;
  int32_t* experts;
  float* weights;
  int32_t* rows;
  int32_t* offsets;
  int* hist;  // [blocks][E + 1]
  int per, blocks;  // tokens per block
  int* err;
};

// A total order of the values as unsigned integers: NaN highest, -0 as +0.
__device__ __forceinline__ uint32_t ordered(float x) {
  if (x != x) return kFull;
  const uint32_t u = __float_as_uint(x + 0.f);
  return u & 0x80000000u ? ~u : u | 0x80000000u;
}

__device__ __forceinline__ float from_ordered(uint32_t u) {
  return __uint_as_float(u & 0x80000000u ? u & 0x7fffffffu : ~u);  // (the NaN pattern gives a NaN)
}

__device__ __forceinline__ float logit(const RouteArgs& a, int t, int e) {
  const size_t i = (size_t)t * a.ld + e, n = span(a.T, a.ld, a.E);
  if (a.type == 2) {
    const float* p = static_cast<const float*>(a.logits);
    return __ldg(ld_at(p + i, p, n, a.err));
  }
  const uint16_t* p = static_cast<const uint16_t*>(a.logits);
  const uint16_t v = __ldg(ld_at(p + i, p, n, a.err));
  return a.type == 1 ? value16<true>(v) : value16<false>(v);
}

template <int V>
__device__ __forceinline__ void load_logits(const RouteArgs& a, int t, int lane, float (&x)[V]) {
#pragma unroll
  for (int i = 0; i < V; ++i) {
    const int e = lane + 32 * i;
    x[i] = e < a.E ? logit(a, t, e) : -INFINITY;
  }
}

// The experts of a token with the logits x (expert lane + 32 i in x[i]): lane
// j < k gets its j-th and writes it with its weight.
template <int V>
__device__ __forceinline__ int choose(const RouteArgs& a, int t, int lane, const float (&x)[V]) {
  uint32_t key[V];
#pragma unroll
  for (int i = 0; i < V; ++i) key[i] = ordered(x[i]);
  int mine = -1;
  float value = 0.f, highest = 0.f;
  for (int j = 0; j < a.k; ++j) {
    uint32_t best = key[0];
#pragma unroll
    for (int i = 1; i < V; ++i) best = max(best, key[i]);
    const uint32_t top = __reduce_max_sync(kFull, best);
    if (top <= kLowest) break;
    uint32_t index = kFull;
#pragma unroll
    for (int i = V - 1; i >= 0; --i)
      if (key[i] == top) index = lane + 32 * i;
    index = __reduce_min_sync(kFull, index);
#pragma unroll
    for (int i = 0; i < V; ++i)
      if ((int)index == lane + 32 * i) key[i] = 0;
    if (j == 0) highest = from_ordered(top);
    if (lane == j) {
      mine = (int)index;
      value = from_ordered(top);
    }
  }
  float score = 0.f, total = 1.f;
  if (a.sigmoid) {
    if (mine >= 0) score = 1.f / (1.f + expf(-value));
  } else {
    if (mine >= 0) score = expf(value - highest);
    if (!a.renormalize) {
      float s = 0.f;
#pragma unroll
      for (int i = 0; i < V; ++i)
        if (lane + 32 * i < a.E) s += expf(x[i] - highest);
#pragma unroll
      for (int d = 16; d; d >>= 1) s += __shfl_xor_sync(kFull, s, d);
      total = s;
    }
  }
  if (a.renormalize) {
    total = score;
#pragma unroll
    for (int d = 16; d; d >>= 1) total += __shfl_xor_sync(kFull, total, d);
  }
  if (lane < a.k) {
    const size_t f = (size_t)t * a.k + lane, n = (size_t)a.T * a.k;
    if (in_buf(a.experts + f, a.experts, n, a.err)) a.experts[f] = mine;
    // (sigmoids that all underflow have no sum to be divided by)
    if (in_buf(a.weights + f, a.weights, n, a.err)) a.weights[f] = mine < 0 || total == 0.f ? 0.f : score / total;
  }
  return mine;
}

// Places the choices [f0, f1) of a block: each warp a contiguous part of
// them. next [kWarps][E + 1], in shared memory, holds the place of each
// warp's next choice of each expert.
__device__ __forceinline__ int expert_of(const RouteArgs& a, int f) {
  const int e = *ld_at(a.experts + f, a.experts, (size_t)a.T * a.k, a.err);
  return e < 0 ? a.E : e;
}
__device__ void place(const RouteArgs& a, int f0, int f1, const int* base, int* next) {
  const int warp = threadIdx.x / 32, lane = threadIdx.x % 32, bins = a.E + 1;
  const int len = ((f1 - f0 + kWarps - 1) / kWarps + 31) / 32 * 32;
  const int g0 = min(f0 + warp * len, f1), g1 = min(g0 + len, f1);
  int* mine = next + warp * bins;
  for (int i = threadIdx.x; i < kWarps * bins; i += kThreads) next[i] = 0;
  __syncthreads();
  for (int f = g0 + lane; f < g1; f += 32) atomicAdd(mine + expert_of(a, f), 1);
  __syncthreads();
  for (int e = threadIdx.x; e < bins; e += kThreads) {
    int at = base[e];
    for (int w = 0; w < kWarps; ++w) {
      const int n = next[w * bins + e];
      next[w * bins + e] = at;
      at += n;
    }
  }
  __syncthreads();
  for (int f = g0; f < g1; f += 32) {
    const bool live = f + lane < g1;
    const int e = live ? expert_of(a, f + lane) : -1;
    const uint32_t same = __match_any_sync(kFull, e);
    const uint32_t before = same & ((1u << lane) - 1);
    int at = 0;
    if (live) at = mine[e] + __popc(before);
    __syncwarp();
    if (live && before == 0) mine[e] += __popc(same);
    __syncwarp();
    if (live && in_buf(a.rows + at, a.rows, (size_t)a.T * a.k, a.err)) a.rows[at] = f + lane;
  }
}

// Exclusive prefix sums of count[0 .. n) in place, by the first warp.
__device__ __forceinline__ void prefix(int* count, int n) {
  if (threadIdx.x >= 32) return;
  int sum = 0;
  for (int i = threadIdx.x; i - (int)threadIdx.x < n; i += 32) {
    const int v = i < n ? count[i] : 0;
    int s = v;
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
      const int u = __shfl_up_sync(kFull, s, d);
      if ((int)threadIdx.x >= d) s += u;
    }
    if (i < n) count[i] = sum + s - v;
    sum += __shfl_sync(kFull, s, 31);
  }
}

__device__ __forceinline__ void write_offsets(const RouteArgs& a, const int* first) {
  for (int e = threadIdx.x; e <= a.E; e += kThreads)
    if (in_buf(a.offsets + e, a.offsets, (size_t)a.E + 1, a.err)) a.offsets[e] = first[e];
}

// Experts and weights of a block's tokens and the counts of its choices
// (hist's row of the block); with kAll the only block, which places them too.
template <int V, bool kAll>
__global__ void __launch_bounds__(kThreads) choose_kernel(const RouteArgs a) {
  extern __shared__ int shared[];  // [E + 1] counts, with kAll [kWarps][E + 1] after them
  const int warp = threadIdx.x / 32, lane = threadIdx.x % 32, bins = a.E + 1;
  allow_dependent_launch();
  for (int i = threadIdx.x; i < bins; i += kThreads) shared[i] = 0;
  __syncthreads();
  grid_dependency_wait();
  const int t0 = blockIdx.x * a.per, t1 = min(t0 + a.per, a.T);
  float x[V], ahead[V];
  if (t0 + warp < t1) load_logits(a, t0 + warp, lane, ahead);
  for (int t = t0 + warp; t < t1; t += kWarps) {
#pragma unroll
    for (int i = 0; i < V; ++i) x[i] = ahead[i];
    if (t + kWarps < t1) load_logits(a, t + kWarps, lane, ahead);
    const int e = choose(a, t, lane, x);
    if (lane < a.k) atomicAdd(shared + (e < 0 ? a.E : e), 1);
  }
  __syncthreads();
  if (kAll) {
    prefix(shared, bins);
    __syncthreads();
    write_offsets(a, shared);
    place(a, 0, a.T * a.k, shared, shared + bins);
  } else {
    int* to = a.hist + (size_t)blockIdx.x * bins;
    for (int i = threadIdx.x; i < bins; i += kThreads)
      if (in_buf(to + i, a.hist, (size_t)a.blocks * bins, a.err)) to[i] = shared[i];
  }
}

// Places a block's choices behind those of lower experts and, of the same
// expert, of earlier blocks.
__global__ void __launch_bounds__(kThreads) place_kernel(const RouteArgs a) {
  extern __shared__ int shared[];  // first [E + 1], before [E + 1], next [kWarps][E + 1]
  const int bins = a.E + 1;
  int *first = shared, *before = shared + bins, *next = before + bins;
  allow_dependent_launch();
  for (int i = threadIdx.x; i < 2 * bins; i += kThreads) shared[i] = 0;
  __syncthreads();
  grid_dependency_wait();
  // the counts' columns, split over as many threads as there are
  const int parts = max(1, kThreads / bins), part = threadIdx.x / bins;
  for (int e = threadIdx.x % bins; part < parts && e < bins; e += kThreads) {
    int all = 0, own = 0;
    constexpr int kFlight = 12;  // counts in flight
    for (int b0 = part; b0 < a.blocks; b0 += parts * kFlight) {
      int n[kFlight];
#pragma unroll
      for (int i = 0; i < kFlight; ++i) {
        const int b = b0 + i * parts;
        n[i] = b < a.blocks ? __ldcg(ld_at(a.hist + (size_t)b * bins + e, a.hist, (size_t)a.blocks * bins, a.err)) : 0;
      }
#pragma unroll
      for (int i = 0; i < kFlight; ++i) {
        all += n[i];
        own += b0 + i * parts < (int)blockIdx.x ? n[i] : 0;
      }
    }
    atomicAdd(first + e, all);
    atomicAdd(before + e, own);
  }
  __syncthreads();
  prefix(first, bins);
  __syncthreads();
  if (blockIdx.x == 0) write_offsets(a, first);
  for (int e = threadIdx.x; e < bins; e += kThreads) before[e] += first[e];
  __syncthreads();
  const int t0 = blockIdx.x * a.per, t1 = min(t0 + a.per, a.T);
  place(a, t0 * a.k, t1 * a.k, before, next);
}

template <int V>
cudaError_t launch_choose(const RouteArgs& a, cudaStream_t stream) {
  const size_t bins = (size_t)(a.E + 1) * sizeof(int);
  if (a.blocks == 1)
    return launch_pdl(choose_kernel<V, true>, dim3(1), dim3(kThreads), (kWarps + 1) * bins, stream, a);
  cudaError_t e = launch_pdl(choose_kernel<V, false>, dim3((unsigned)a.blocks), dim3(kThreads), bins, stream, a);
  if (e != cudaSuccess) return e;
  return launch_pdl(place_kernel, dim3((unsigned)a.blocks), dim3(kThreads), (kWarps + 2) * bins, stream, a);
}

int tokens_per_block(int T) {
  if (T <= kOneBlock) return T;
  const int per = (T + kBlocks - 1) / kBlocks;
  return per < kWarps ? kWarps : per;
}

}  // namespace

size_t route_workspace_bytes(int T, int E) {
  if (T <= kOneBlock) return 0;
  const int per = tokens_per_block(T);
  return kWorkspaceFlags + (size_t)((T + per - 1) / per) * (E + 1) * sizeof(int);
}

cudaError_t launch_route(const void* logits, long long ld, int type, int T, int E, int k, bool sigmoid,
                         bool renormalize, int32_t* experts, float* weights, int32_t* rows, int32_t* offsets,
                         void* workspace, cudaStream_t stream) {
  const int per = T > 0 ? tokens_per_block(T) : 0;
  RouteArgs a = {logits, ld, type, T, E, k, sigmoid, renormalize, experts, weights, rows, offsets,
                 workspace ? reinterpret_cast<int*>(static_cast<uint8_t*>(workspace) + kWorkspaceFlags) : nullptr,
                 per, T > 0 ? (T + per - 1) / per : 1, nullptr};
  cudaError_t e = device_error_word(&a.err);
  if (e != cudaSuccess) return e;
  if (E <= 32) return launch_choose<1>(a, stream);
  if (E <= 64) return launch_choose<2>(a, stream);
  if (E <= 128) return launch_choose<4>(a, stream);
  if (E <= 256) return launch_choose<8>(a, stream);
  return launch_choose<16>(a, stream);
}

}  // namespace w4a16
