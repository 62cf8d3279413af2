// W4A16 products grouped by expert on the tensor cores (sm_103a:
// tcgen05.mma.cta_group::2, tensor memory, TMA), for many rows per expert.
//
// Choice f of expert e: Y[f][n] = sum_k A[f or f / top][k] W_e[k][n], with the
// gate/up epilogue silu(gate) * up of columns [gate | up], or the products
// rounded to 16 bits for the weighted sum over a token's choices
// (experts.cu forms it in fp32).
//
// The contraction is the one of the kernel for one weight (tc_pair.cu): a
// cluster of two CTAs makes a tile of 256 weight columns, each CTA dequantizing
// its 128 columns, RNE((q - z) s) in the activations' type, straight into
// tensor memory (the MMA's A operand) and staging half of the rows (the B
// operand). What differs:
//   - A tile has up to 256 rows in one or two parts of up to 128, each with
//     its own accumulator. An expert's n rows make ceil(n / 256) tiles of the
//     same size, and the MMA's N is a part's size, rounded up to 16: an expert
//     of 40 rows costs MMAs of 48. Which tiles there are is known on the device
//     only: every CTA makes the list of the experts' first tiles from the
//     offsets when it starts, and each role walks it (a cluster's tiles
//     ascend).
//   - The rows are gathered by the converting warps: while a group converts
//     a stage it copies the stage's rows (cp.async, eight lanes a row of 128
//     bytes, to the swizzled places), and each of its warps waits for its own
//     copies before it arrives for the stage. (tile::gather4 copies by the lanes
//     of one warp took about 95 cycles each, one warp's cp.async about 85: the
//     MMAs waited for rows most of the time.) Places beyond a tile's rows repeat
//     its last row; their results are not stored.
//   - With silu(gate) * up a CTA's eight strips are four of gate columns and
//     the four of up columns beside them (one 4-D copy), placed so that of a
//     warp's tensor-memory lanes 0..15 hold gate and 16..31 up of the same 16
//     results: read 16 lanes at a time, a thread gets both of a result in fp32,
//     and the output is half as wide.
//   - K is short (an expert's inner width), so that a tile's end matters: the
//     converting warps hand the first part's accumulator back before they take
//     the second's, and the next tile begins with the first part's MMAs of the
//     stages that are converted already, to catch up with the second part's
//     when its accumulator is free.
// What bounds it is the converting warps: a stage takes one of them (four run
// on a scheduler) about 600 instructions, so that a stage is two atoms (of the
// last one only what K has), tiles are found without divisions, and hardly a
// register is spilled: the first-level cache beside 223 KB of shared memory is
// too small for that, and each spilled value cost a trip to L2 (519 -> 336 us at
// the first case below).
// Measured (us a call, TFLOP/s): 4099 tokens, 64 experts, top 8, gate and up of
// 2048 x 2048, bf16 235, 1170; down of 1024 x 2048 with the sum 169, 815; 2047
// tokens, 8 experts, top 2, down of 11008 x 4096 with the sum 286-293, 1260-1290 (of
// it 24% an SM's wait for the last round of tiles: 3.4 tiles to a cluster make
// four rounds).
//
// Rings, barriers and their invariants are those of tc_pair.cu, without a
// barrier for the rows' arrival. What a group waits for before it converts stage
// s are the MMAs of stages s - 5 (the rows' slot) and s - 4 (the dequantized
// slot), which need no accumulator that the group has still to hand back. Every
// wait is bounded; a wait that gives up sets the library's error word, and its
// CTA drains and leaves through the same final cluster barrier as a normal run.
#include <cuda.h>
#include <cudaTypedefs.h>

#include "experts.cuh"
#include "tc_pair.cuh"

namespace w4a16 {
namespace {

using namespace tc;
using namespace pair;

constexpr int kGroups = 4;                  // dequantizing groups of four warps
constexpr int kFirst = 2;                   // the first converting warp, after producer and MMA issuer
constexpr int kThreads = 32 * kFirst + 128 * kGroups;
constexpr int kRows = 128;                  // most rows of a part (MMA N); a tile has two
constexpr int kAtoms = 2;                   // 64-k atoms of a stage
constexpr int kPartSlot = kRows / 2 * 128;  // bytes of a CTA's rows of one atom of a part, at most
constexpr int kAtomSlot = 2 * kPartSlot;
constexpr int kActSlot = kAtoms * kAtomSlot;
constexpr int kCodeSlot = kAtoms * kCodeAtomBytes;
constexpr int kMostExperts = 512;
constexpr float kHalfInfinite = 65520.f;  // the least that rounds to fp16's infinity
constexpr uint32_t kHalfInf = 0x7c00u;    // which is

struct TensorParams {
  ExpertArgs a;
  uint16_t* D;     // combined: [choices][N], the products
  float* wide;     // the same in fp32, written where fp16 products are infinite
  int pairs;       // tiles along the columns
  float inv_group;  // 1 / group
};

// Tile t of the launch (which lies in expert e's): 256 columns (with silu 128
// of gate and of up) x the rows [first, first + n) of the list, in `parts` parts
// of `size` (the MMA's N).
struct Tile {
  int e, col, first, n, parts, size;
};

// Ring depths per CTA: the dequantized operand in the tensor memory beside the
// accumulators, four slots, one per group; codes four; the rows five.
constexpr int kActSlots = 5, kCodeSlots = 4, kDqSlots = (512 - 2 * kRows) / (kAtoms * kAtomCols);
static_assert(kDqSlots == kGroups && kCodeSlots == kGroups && kActSlots == kGroups + 1, "slots by the group's number");
constexpr int kMetaBytes = 128 * kGroups * 8 * kAtoms;  // scales and zero points of every converting thread
constexpr int kSmemBytes = kActSlots * kActSlot + kCodeSlots * kCodeSlot + 1024 + kBarBytes + kMetaBytes + 4 * kGroups * 1024;  // (a staged chunk per warp)
static_assert(kSmemBytes + 14 * kMostExperts + 64 <= kSmemLimit && 8 * (kActSlots + kDqSlots + 2 * kCodeSlots + 5) + 8 <= kBarBytes, "shared memory");

__device__ __forceinline__ int row_tiles(int n) { return (n + 2 * kRows - 1) / (2 * kRows); }

// 4-D tile load (x innermost).
__device__ __forceinline__ void tma_load_4d(uint32_t dst, const CUtensorMap* map, int x, int y, int z, int w,
                                            uint32_t bar) {
  asm volatile(
      "cp.async.bulk.tensor.4d.shared::cluster.global.mbarrier::complete_tx::bytes"
      " [%0], [%1, {%2, %3, %4, %5}], [%6];" ::"r"(dst),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(x), "r"(y), "r"(z), "r"(w), "r"(bar)
      : "memory");
}

// copy16 where `ok`, without a branch.
__device__ __forceinline__ void copy16_if(bool ok, uint32_t to, const void* from) {
  asm volatile("{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %2, 0;\n\t@p cp.async.cg.shared.global [%0], [%1], 16;\n\t}" ::"r"(to),
               "l"(from), "r"((int)ok)
               : "memory");
}
// One lane of a converged warp.
__device__ __forceinline__ bool elect_one() {
  uint32_t ok;
  asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.u32 %0, 1, 0, p;\n\t}" : "=r"(ok));
  return ok != 0;
}
// all of this thread's copies have landed
__device__ __forceinline__ void copies_wait() { asm volatile("cp.async.wait_all;" ::: "memory"); }

// 16 lanes of tensor memory x 16 columns: r[4 m + 2 v + c] is lane (thread / 4 +
// 8 v), column 8 m + 2 (thread % 4) + c.
__device__ __forceinline__ void tmem_ld_16x16(uint32_t taddr, uint32_t (&r)[8]) {
  asm volatile("tcgen05.ld.sync.aligned.16x256b.x2.b32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7])
               : "r"(taddr));
}
// Of each pair of fp16 the larger in magnitude (a number beside NaN), of either sign.
__device__ __forceinline__ uint32_t max_abs2(uint32_t a, uint32_t b) {
  uint32_t d;
  asm("max.xorsign.abs.f16x2 %0, %1, %2;" : "=r"(d) : "r"(a), "r"(b));
  return d;
}
// Four 8x8 matrices of 16-bit values, stored transposed: thread 8 i + j gives
// where matrix i's column j goes, as a row of 16 bytes.
__device__ __forceinline__ void stmatrix_trans(uint32_t at, const uint32_t (&m)[4]) {
  asm volatile("stmatrix.sync.aligned.m8n8.x4.trans.shared.b16 [%0], {%1, %2, %3, %4};" ::"r"(at), "r"(m[0]), "r"(m[1]), "r"(m[2]),
               "r"(m[3])
               : "memory");
}

// The bf16 dequantization of one column, RNE((q - z) s) as dequant_word_bf16
// gives it, in pairs: q - z is exact in bf16, and with s = hi + lo, hi its
// rounding to bf16 and lo the remaining (at most three) bits, (q - z) lo is
// exact too, so that one fma of exact operands rounds the exact product once.
// Four instructions a pair instead of five.
struct DeqSplitBf16 {
  __nv_bfloat162 zero, hi, lo;  // 128 + z, and the parts of the scale
  __device__ __forceinline__ DeqSplitBf16(uint32_t z, uint16_t s_bits) {
    const uint32_t b = 0x43004300u | z | (z << 16);
    zero = *reinterpret_cast<const __nv_bfloat162*>(&b);
    const float s = __half2float(__ushort_as_half(s_bits));
    const __nv_bfloat16 h = __float2bfloat16_rn(s);
    hi = __bfloat162bfloat162(h);
    lo = __bfloat162bfloat162(__float2bfloat16_rn(s - __bfloat162float(h)));
  }
  __device__ __forceinline__ void word(uint32_t w, uint32_t* out) const {
    const uint32_t t = w & 0x0F0F0F0Fu, u = (w >> 4) & 0x0F0F0F0Fu;
    const uint32_t x[4] = {__byte_perm(t, 0x43434343u, 0x4240), __byte_perm(t, 0x43434343u, 0x4341),
                           __byte_perm(u, 0x43434343u, 0x4240), __byte_perm(u, 0x43434343u, 0x4341)};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const __nv_bfloat162 d = __hsub2(*reinterpret_cast<const __nv_bfloat162*>(&x[i]), zero);
      const __nv_bfloat162 v = __hfma2(d, hi, __hmul2(d, lo));
      out[i] = *reinterpret_cast<const uint32_t*>(&v);
    }
  }
};

template <bool kB>
__global__ void __launch_bounds__(kThreads, 1)
experts_tc_kernel(const __grid_constant__ CUtensorMap tmW, const TensorParams p) {
  extern __shared__ uint8_t smem_raw[];
  const ExpertArgs& a = p.a;
  // the same offsets in both CTAs: the MMA's descriptors, given by the first
  // CTA, address the second CTA's operands at the same shared addresses
  const uint32_t raw = (uint32_t)__cvta_generic_to_shared(smem_raw);
  const uint32_t base = (raw + 1023u) & ~1023u;
  constexpr int nact = kActSlots, ncode = kCodeSlots, ndq = kDqSlots;
  constexpr uint32_t kActBytes = kActSlot, kCodeBytes = kCodeSlot;
  constexpr int kDqCol0 = 2 * kRows;  // tensor memory: two accumulators, then the dequantized operand
  // [activation ring | code ring | barriers | scales | staged results], 1024-aligned slots
  const uint32_t code_base = base + (uint32_t)nact * kActBytes;
  const uint32_t bars = code_base + (uint32_t)ncode * kCodeBytes;
  auto stage_done = [&](int i) { return bars + 8u * i; };
  auto dq_full = [&](int i) { return bars + 8u * (nact + i); };
  auto code_full = [&](int i) { return bars + 8u * (nact + ndq + i); };
  auto code_empty = [&](int i) { return bars + 8u * (nact + ndq + ncode + i); };
  // of a part's accumulator
  auto accum_full = [&](int part) { return bars + 8u * (nact + ndq + 2 * ncode + part); };
  auto accum_empty = [&](int part) { return bars + 8u * (nact + ndq + 2 * ncode + 2 + part); };  // used in the first CTA
  const uint32_t drain_bar = bars + 8u * (nact + ndq + 2 * ncode + 4);  // the MMAs issued before an abort completed
  const uint32_t tmem_slot = drain_bar + 8u;
  uint8_t* gen_base = smem_raw + (base - raw);
  // (fixed places, which take no registers)
  __shared__ int abort_word, offs[kMostExperts + 1];  // [E + 1]
  __shared__ int firsts[kMostExperts + 1];            // [E + 1]: an expert's first tile
  __shared__ float inverse[kMostExperts];             // of an expert's row tiles
  __shared__ short sizes[kMostExperts];               // of its parts; negative: a tile has one
  volatile int* abort_flag = &abort_word;

  const uint32_t rank = cluster_rank();  // 0: the CTA that issues the MMAs
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int cluster = blockIdx.x >> 1, clusters = gridDim.x >> 1;
  const int natoms = a.K / kStageK, nk = (natoms + kAtoms - 1) / kAtoms;  // stages of one tile

  if (threadIdx.x == 0) {
    for (int i = 0; i < nact; ++i) mbar_init(stage_done(i), 1);
    for (int i = 0; i < ndq; ++i) mbar_init(dq_full(i), 8);  // used in the first CTA: a group of both CTAs
    for (int i = 0; i < ncode; ++i) {
      mbar_init(code_full(i), 1);
      mbar_init(code_empty(i), 4);  // the warps of the group that converts the stage
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(accum_full(i), 1);
      mbar_init(accum_empty(i), 2 * 4 * kGroups);  // every dequant warp of both CTAs
    }
    mbar_init(drain_bar, 1);
    *abort_flag = 0;
    fence_barrier_init();
  }
  if (warp == 1) {
    pair_tmem_alloc(tmem_slot, 512);
    pair_tmem_relinquish();
  }
  grid_dependency_wait();
  for (int e = threadIdx.x; e <= a.E; e += kThreads) offs[e] = offset_of(a, e);
  __syncthreads();
  if (warp == 0) {
    // the list: offsets that never decrease (recorded where they do), and the
    // prefix sums of the experts' tiles
    int top = 0, sum = 0;
    for (int e0 = 0; e0 <= a.E; e0 += 32) {
      const int e = e0 + lane;
      const int v = e <= a.E ? offs[e] : 0;
      int m = max(v, top);
#pragma unroll
      for (int d = 1; d < 32; d <<= 1) {
        const int u = __shfl_up_sync(0xffffffffu, m, d);
        if (lane >= d) m = max(m, u);
      }
      if (e <= a.E) {
        if (m != v) atomicOr(a.err, kErrRange);
        offs[e] = m;
      }
      // the tiles of expert e - 1, which ends here
      int before = __shfl_up_sync(0xffffffffu, m, 1);
      if (lane == 0) before = top;
      int s = e > 0 && e <= a.E ? row_tiles(m - before) * p.pairs : 0;
      if (s > 0) {
        const int rt = row_tiles(m - before), each = (m - before + rt - 1) / rt;
        inverse[e - 1] = 1.f / (float)rt;
        sizes[e - 1] = (short)(each > kRows ? ((each + 1) / 2 + 15) & ~15 : -((each + 15) & ~15));
      }
#pragma unroll
      for (int d = 1; d < 32; d <<= 1) {
        const int u = __shfl_up_sync(0xffffffffu, s, d);
        if (lane >= d) s += u;
      }
      if (e <= a.E) firsts[e] = sum + s;
      sum += __shfl_sync(0xffffffffu, s, 31);
      top = __shfl_sync(0xffffffffu, m, 31);
    }
  }
  tc_fence_before();
  cluster_sync();  // both CTAs' barriers initialized, tensor memory allocated, lists made
  tc_fence_after();
  const uint32_t tmem_base = *reinterpret_cast<volatile uint32_t*>(gen_base + (tmem_slot - base));
  allow_dependent_launch();

  // this cluster's tiles: cluster, cluster + clusters, ...
  const int tiles = firsts[a.E];
  const int ntl = cluster < tiles ? (tiles - 1 - cluster) / clusters + 1 : 0;
  const int total = ntl * nk;  // stages of the cluster's sequence
  // tile i of the sequence; e: of a tile before it (0 at first), moved on
  auto tile_at = [&](int i, int& e) -> Tile {
    const int t = cluster + i * clusters;
    while (firsts[e + 1] <= t) ++e;
    // (row tiles fastest; the quotient by their number as a product with its
    // inverse, which is exact below 2^21: the next integer is at least half an
    // inverse away, the product's error less)
    const int n = offs[e + 1] - offs[e], rt = row_tiles(n), local = t - firsts[e];
    const int col = local < 1 << 21 ? (int)(((float)local + 0.5f) * inverse[e]) : local / rt;
    const int signed_size = sizes[e], size = abs(signed_size), parts = signed_size > 0 ? 2 : 1;
    const int row = (local - col * rt) * parts * size;
    return {e, col, offs[e] + row, min(parts * size, n - row), parts, size};
  };
  // the first strip of this CTA in a tile (with silu: of its gate columns)
  auto first_strip = [&](const Tile& t) { return (2 * t.col + (int)rank) * (a.silu ? 4 : 8); };

  if (warp == 0) {
    // ---------------------------------------------------------- producer
    // one thread keeps the code ring full
    if (lane == 0 && total > 0) {
      int e = 0, s = 0;
      SeqPos seq{0, 0};
      RingPos pos{0, 0u};
      Tile t = tile_at(0, e);
      for (; s < total; ++s) {
        if (s >= ncode && !mbar_wait(code_empty(pos.slot), pos.phase ^ 1u, abort_flag, kErrProducer, a.err)) break;
        const uint32_t to = code_base + (uint32_t)pos.slot * kCodeBytes;
        if (in_smem(to, kCodeBytes, raw, a.err)) {
          mbar_expect_tx(code_full(pos.slot), kCodeBytes);
          tma_load_4d(to, &tmW, 0, seq.kb * kAtoms * 4, first_strip(t), a.silu ? 2 * t.e : t.e, code_full(pos.slot));
        }
        pos.step(1, ncode);
        const int tl = seq.tile;
        seq.step(1, nk);
        if (seq.tile != tl && s + 1 < total) t = tile_at(seq.tile, e);
      }
      if (*abort_flag) {
        // let the copies already issued land before the CTA leaves
        for (int i = (s > ncode ? s - ncode : 0); i < s; ++i)
          mbar_drain(code_full(i % ncode), (uint32_t)(i / ncode) & 1u, a.err);
      } else {
        // the pair's last commits have reached this CTA: none is still on its way
        for (int i = (total > nact ? total - nact : 0); i < total; ++i)
          if (!mbar_wait_poll(stage_done(i % nact), (uint32_t)(i / nact) & 1u, abort_flag, kErrProducer, a.err)) break;
      }
    }
  } else if (warp == 1) {
    if (rank == 0 && total > 0 && elect_one()) {
      // ---------------------------------------------------------- MMA issuer (first CTA)
      // (an elected lane of a converged warp: the operands' places then stay in
      // uniform registers, and an MMA takes few instructions to issue)
      // stage n of the sequence has dequantized slot n & 3, and `slot` of the rows
      const uint64_t bdesc0 = sw128_kmajor_desc(base);
      int n = 0, slot = 0;
      auto after = [&](int k) { return k + 1 == nact ? 0 : k + 1; };
      int e = 0;
      bool ok = true;
      for (int tl = 0; tl < ntl && ok; ++tl) {
        const Tile t = tile_at(tl, e);
        const uint32_t idesc = f16_idesc(2 * kCols, t.size, kB);
        const uint32_t phase = (uint32_t)(tl - 1) & 1u;  // of the accumulators' release by the tile before
        auto ready = [&](int i) {
          return mbar_wait_poll(dq_full(i & 3), (uint32_t)(i >> 2) & 1u, abort_flag, kErrMma, a.err);
        };
        // the MMAs (16 k each: 8 columns of A, 32 bytes of B) of a part of
        // stage i, whose rows are in slot k
        auto mmas = [&](int i, int k, int part, int kb) {
#pragma unroll
          for (int u = 0; u < kAtoms; ++u) {
            if (kb * kAtoms + u >= natoms) break;
            const uint32_t place = (uint32_t)(k * kActSlot + u * kAtomSlot + part * kPartSlot);
            const uint32_t acol = (uint32_t)(kDqCol0 + ((i & 3) * kAtoms + u) * kAtomCols);
            if (!in_smem(base + place, kPartSlot, raw, a.err) || !in_tmem(acol, kAtomCols, 512, a.err)) return;
            const uint64_t bdesc = bdesc0 + (place >> 4);
#pragma unroll
            for (int kk = 0; kk < kStageK / 16; ++kk)
              pair_mma_f16_ts(tmem_base + (uint32_t)(part * kRows), tmem_base + acol + (uint32_t)(8 * kk), bdesc + 2u * kk,
                              idesc, (kb | u | kk) != 0);
          }
        };
        if (tl > 0 && !(ok = mbar_wait_poll(accum_empty(0), phase, abort_flag, kErrMma, a.err))) break;
        // after another tile, the first part of the stages that there are slots
        // for, then the second (no slot is freed in between)
        const int begin = tl > 0 && t.parts == 2 ? min(nk, ndq) : 0;
        for (int kb = 0, k = slot; kb < begin && ok; ++kb, k = after(k)) {
          if (!(ok = ready(n + kb))) break;
          tc_fence_after();
          mmas(n + kb, k, 0, kb);
        }
        if (ok && begin == nk) pair_commit_both(accum_full(0));
        if (ok && tl > 0) ok = mbar_wait_poll(accum_empty(1), phase, abort_flag, kErrMma, a.err);
        for (int kb = 0; kb < begin && ok; ++kb, ++n, slot = after(slot)) {
          mmas(n, slot, 1, kb);
          pair_commit_both(stage_done(slot));
        }
        for (int kb = begin; kb < nk && ok; ++kb, ++n, slot = after(slot)) {
          if (!(ok = ready(n))) break;
          tc_fence_after();
          mmas(n, slot, 0, kb);
          if (kb + 1 == nk) pair_commit_both(accum_full(0));
          if (t.parts == 2) mmas(n, slot, 1, kb);
          pair_commit_both(stage_done(slot));
        }
        if (ok) pair_commit_both(accum_full(1));
      }
      if (!ok) {
        // no MMA may run past the release of tensor memory: one more commit,
        // to both CTAs' drain barriers, fires once every MMA issued has completed
        pair_commit_both(drain_bar);
        mbar_drain(drain_bar, 0, a.err);
      }
    }
  } else {
    // ---------------------------------------------------------- dequant + epilogue
    // Group g converts the stages g, g + groups, ... of the cluster's
    // sequence. Thread (lane quarter q, lane) owns tensor-memory lane 32 q +
    // lane: column c = lane % 16 of the CTA's strip 2 q + lane / 16 (with silu:
    // of gate strip q, or up strip q, the CTA's strip 4 + q).
    const int dw = warp - kFirst;
    const int grp_id = dw >> 2;
    const int q = warp & 3;
    const int ls = a.silu ? q + 4 * (lane >> 4) : 2 * q + (lane >> 4);
    const int c = lane & 15, cp = c & 7;
    const bool hi = c >= 8;
    const int G = a.K / a.group, strips = a.N / kStripCols;
    const int limit = a.silu ? strips / 2 : strips;  // strips of an expert's (half) columns
    const uint32_t tlane = (uint32_t)(32 * q) << 16;
    const int width = a.silu ? a.N / 2 : a.N;

    // choices of no expert: zeros
    if (!a.combine)
      for (int i = offs[a.E] + (int)blockIdx.x; i < choices(a); i += gridDim.x) {
        const int f = choice_of(a, i);
        for (int n = threadIdx.x - 32 * kFirst; f >= 0 && n < width; n += 128 * kGroups) {
          uint16_t* y = a.Y + (size_t)f * width + n;
          if (in_buf(y, a.Y, (size_t)choices(a) * width, a.err)) *y = 0;
        }
      }

    const uint32_t dq_remote = cluster_addr(dq_full(grp_id), 0);       // the first CTA's dq_full of this group's slot
    // a wait that every lane of the warp passes or every lane gives up on:
    // the tensor-memory stores and loads that follow are .sync.aligned
    auto warp_wait = [&](uint32_t bar, uint32_t parity, bool poll, int code) -> bool {
      const bool ok = poll ? mbar_wait_poll(bar, parity, abort_flag, code, a.err)
                           : mbar_wait(bar, parity, abort_flag, code, a.err);
      return __all_sync(0xffffffffu, ok);
    };

    // The group's stages are s = grp_id, grp_id + 4, ...: they have the code
    // slot and the dequantized slot grp_id, and the slot s % 5 of the rows. `next`
    // is the next stage to fetch rows and scales for: its place, its tile's
    // expert, this lane's strip of all experts' strips (-1: beyond the columns),
    // the group of its first scale, and the rows.
    SeqPos next{grp_id, 0};
    next.step(0, nk);
    constexpr int kStep = kAtoms * kStageK;  // k of a stage
    int ne = 0, nstrip = -1, ngrp = 0;
    // (k / group, exact below 2^21 as above)
    auto group_of = [&](int kb) { return (int)(((float)(kb * kStep) + 0.5f) * p.inv_group); };
    const bool one_group = a.group % kStep == 0;  // of both atoms of a stage
    // Rows: of each part this warp copies those of steps q, q + 4, ... (step
    // i: rows 4 i .. 4 i + 3 of this CTA's half of it), a lane the 16 bytes lane
    // % 8 of row lane / 8 of each; lane 16 part + 4 j + r holds which row of A
    // is the r-th of the warp's j-th step of the part.
    constexpr int kSteps = kRows / 2 / 16;
    static_assert(2 * 4 * kSteps == 32, "a row per lane");
    int held = 0, half = 0;  // half: of a part's rows; minus that with one part
    auto enter_tile = [&]() {
      const Tile t = tile_at(next.tile, ne);
      const int st = first_strip(t) + (a.silu ? q : ls);
      nstrip = st < limit ? t.e * strips + st + (a.silu && lane >= 16 ? limit : 0) : -1;
      half = t.size / 2;
      const int i = min(4 * (q + lane % 16 / 4 * 4) + lane % 4, half - 1);
      const int f = choice_of(a, t.first + min(lane / 16 * t.size + (int)rank * half + i, t.n - 1));
      held = f < 0 ? 0 : a.per_choice ? f : f / a.top;
      if (t.parts == 1) half = -half;
    };
    // the lane's scale and zero point words of its group's next stage, in shared
    // memory: per atom the scales of columns cp and cp + 8, and the zero points of
    // columns cp & 4 .. (cp & 4) + 3, each with its column + 8
    const uint32_t meta = bars + kBarBytes + (uint32_t)(dw * 32 + lane) * 16u;
    auto copy_meta = [&]() {
      if (nstrip < 0) return;
      const uint32_t* sp = reinterpret_cast<const uint32_t*>(a.Sp);
      // (strips times groups are below 2^32: 16 * 64 weights each, in 280 GB)
      uint32_t pg = (uint32_t)nstrip * (uint32_t)G + (uint32_t)ngrp;
#pragma unroll
      for (int u = 0; u < kAtoms; ++u) {
        if (u > 0 && (one_group || next.kb * kAtoms + u >= natoms)) break;
        if (u > 0 && next.kb * kStep + u * kStageK >= (ngrp + 1) * a.group) ++pg;
        copy4(meta + 8u * u, ld_at(sp + (uint64_t)pg * 8u + cp, sp, (size_t)G * a.N * a.E / 2, a.err));
        copy4(meta + 8u * u + 4u, ld_at(a.Zp + (uint64_t)pg * 2u + cp / 4, a.Zp, (size_t)G * a.N * a.E / 8, a.err));
      }
    };
    // chunk lane % 8 of row lane / 8 of a step, swizzled by the row's number in
    // its group of eight: 4 (i & 1) + lane / 8, and i is as odd as q
    const uint32_t place = (uint32_t)q * 512u + (uint32_t)(lane / 8) * 128u +
                           (uint32_t)((lane % 8) ^ (lane / 8 + 4 * (q & 1))) * 16u;
    // (both atoms of) the warp's j-th step of a part, to the stage's slot
    auto copy_step = [&](int part, int j, uint32_t to, const char* from) {
      const uint32_t row = (uint32_t)__shfl_sync(0xffffffffu, held, 16 * part + 4 * j + lane / 8);
      const uint32_t dst = to + (uint32_t)part * kPartSlot + 2048u * j;
      const uint16_t* src = reinterpret_cast<const uint16_t*>(from + (uint64_t)row * (2u * (uint32_t)a.K));
      const bool ok = 4 * (q + 4 * j) < (part == 1 ? half : abs(half)) && in_smem(dst, kAtomSlot + 16, raw, a.err);
      const bool two = ok && (next.kb + 1) * kAtoms <= natoms;
      copy16_if(ok, dst, ok ? ld_at(src, a.A, a_elements(a) - 7, a.err) : src);
      copy16_if(two, dst + kAtomSlot, two ? ld_at(src + kStageK, a.A, a_elements(a) - 7, a.err) : src);
    };
    // Converts the group's it-th stage, stage s of the sequence (whose place is
    // `next`), and copies its rows meanwhile, a few copies between the words of
    // the codes: on their own they would hold the warp up.
    auto stage = [&](int it, int slot) -> bool {
      const int s = grp_id + it * kGroups;
      // the slot's rows, of stage s - 5, have been multiplied
      if (s >= nact && !warp_wait(stage_done(slot), (uint32_t)(s / nact - 1) & 1u, true, kErrDequant)) return false;
      if (!warp_wait(code_full(grp_id), (uint32_t)it & 1u, false, kErrDequant)) return false;
      copies_wait();  // the scales
      const uint32_t cb = code_base + (uint32_t)grp_id * kCodeBytes;
      const uint32_t to = base + (uint32_t)slot * kActBytes + place;
      const char* from = reinterpret_cast<const char*>(a.A + next.kb * kStep + lane % 8 * 8);
#pragma unroll
      for (int u = 0; u < kAtoms; ++u) {
        uint32_t wl[4], wh[4];  // k-octets l and 4 + l
        const uint32_t row = (uint32_t)(ls * 4 * kAtoms + 4 * u + (cp >> 1));  // 128-byte row of the tile
#pragma unroll
        for (int l = 0; l < 4; ++l) {
          const uint32_t chunk = ((uint32_t)(4 * (cp & 1) + l)) ^ (row & 7u);  // 128-byte swizzle
          const uint32_t at = cb + row * 128u + (chunk << 4);
          const uint4 v = lds128(in_smem(at, 16, raw, a.err) ? at : cb);
          wl[l] = hi ? v.y : v.x;
          wh[l] = hi ? v.w : v.z;
        }
        uint32_t sw, zw;
        asm volatile("ld.shared.v2.u32 {%0, %1}, [%2];" : "=r"(sw), "=r"(zw) : "r"(one_group ? meta : meta + 8u * u) : "memory");
        if (u + 1 == kAtoms) {  // the codes are in registers
          __syncwarp();
          if (lane == 0) mbar_arrive(code_empty(grp_id));
        }
        const uint32_t z = (zw >> (8 * (cp & 3) + (hi ? 4 : 0))) & 15u;
        const uint16_t sc = (uint16_t)(sw >> (hi ? 16 : 0));
        uint32_t r[32];  // cell j = (deq[2j], deq[2j + 1]): k-octet o fills cells 4o..4o+3
        if (kB) {
          const DeqSplitBf16 dc(z, sc);
#pragma unroll
          for (int l = 0; l < 4; ++l) {
            dc.word(wl[l], r + 4 * l);
            dc.word(wh[l], r + 16 + 4 * l);
            copy_step(u, l, to, from);
          }
        } else {
          const DeqConst dc = make_deq_const(z, sc);
#pragma unroll
          for (int l = 0; l < 4; ++l) {
            uint32_t o[4];
            dequant_word(wl[l], dc, o);
#pragma unroll
            for (int j = 0; j < 4; ++j) r[4 * l + j] = o[j];
            dequant_word(wh[l], dc, o);
#pragma unroll
            for (int j = 0; j < 4; ++j) r[16 + 4 * l + j] = o[j];
            copy_step(u, l, to, from);
          }
        }
        // the slot's MMAs, of the group's stage before, are done (waited for with
        // the first cells in registers)
        if (u == 0 && it > 0) {
          // (its rows' slot: (s - 4) % 5)
          if (!warp_wait(stage_done(slot + 1 == nact ? 0 : slot + 1), (uint32_t)(s - kGroups) / nact & 1u, true, kErrDequant))
            return false;
          tc_fence_after();
        }
        const uint32_t col = (uint32_t)(kDqCol0 + (grp_id * kAtoms + u) * kAtomCols);
        if (in_tmem(col, kAtomCols, 512, a.err)) tmem_st32(tmem_base + tlane + col, r);
      }
      copies_wait();      // this warp's rows of the stage (the MMAs read them too)
      tmem_wait_st();
      fence_async_shared();  // (the copies wrote them through the generic proxy)
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive_remote(dq_remote);
      return true;
    };
    // this warp's part of tile i's epilogue: tensor-memory lanes 32q..32q+31
    // are this CTA's columns, an accumulator's columns the rows of a part, 16
    // at a time by the groups in turn. A chunk of 16 rows is read as 16 lanes x 8
    // columns per register quad, the layout of an mma.sync result: with silu a
    // thread then has gate and up of the same results. Rounded, it goes through
    // this warp's kilobyte of shared memory, transposed (stmatrix), so that a
    // lane stores 16 bytes of a row.
    constexpr int kChunks = kRows / 16 / kGroups;
    int ee = 0;
    auto epilogue = [&](int i) -> bool {
      uint16_t* out = a.combine ? p.D : a.Y;
      const size_t all = (size_t)choices(a) * width - 7;
      const uint32_t pitch = 2u * (uint32_t)width;  // bytes of a result's row
      const uint32_t stage0 = bars + kBarBytes + kMetaBytes + (uint32_t)dw * 1024u;
      const Tile t = tile_at(i, ee);
      const int s0 = first_strip(t) + (a.silu ? q : 2 * q);  // the warp's first strip of results
#pragma unroll 1
      for (int part = 0; part < 2; ++part) {
        const int n = part < t.parts ? min(t.size, t.n - part * t.size) : 0;
        // the choices of the warp's chunks, on their way while it waits: lane l
        // holds row l of the first chunk, lane 16 + l that of the second
        static_assert(kChunks == 2, "a row per lane");
        const int k = 16 * (grp_id + lane / 16 * kGroups) + lane % 16;
        int chosen = -1;
        if (k < n) chosen = *ld_at(a.rows + t.first + part * t.size + k, a.rows, (size_t)choices(a), a.err);
        if (!warp_wait(accum_full(part), (uint32_t)i & 1u, true, kErrEpilogue)) return false;
        tc_fence_after();
        if (k < n && (unsigned)chosen >= (unsigned)choices(a)) {  // (as choice_of)
          atomicOr(a.err, kErrRange);
          chosen = -1;
        }
#pragma unroll 1
        for (int j = 0; j < kChunks; ++j) {
          const int row0 = 16 * (grp_id + j * kGroups);
          const uint32_t col = (uint32_t)(part * kRows + row0);
          uint32_t r[2][8];  // lanes 0..15, 16..31 of the quarter
          if (row0 < n && in_tmem(col, 16, kDqCol0, a.err)) {
            tmem_ld_16x16(tmem_base + tlane + col, r[0]);
            tmem_ld_16x16(tmem_base + tlane + (16u << 16) + col, r[1]);
          }
          tmem_wait_ld();
          if (j + 1 == kChunks) {  // the warp has read all it reads of this accumulator
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive_remote(cluster_addr(accum_empty(part), 0));  // the first CTA's
          }
          if (row0 >= n) continue;
          // r[j][h][4 m + 2 v + c]: column lane / 4 + 8 v of the strip, row 8 m + 2 (lane % 4) + c
          uint32_t o[2][4];  // rounded: pairs of rows, [strip][2 m + v]
          auto f = [&](int h, int x) { return __uint_as_float(r[h][x]); };
#pragma unroll
          for (int x = 0; x < 4; ++x) {
            if (a.silu) {
              o[0][x] = to_out2<kB>(silu_times(f(0, 2 * x), f(1, 2 * x)), silu_times(f(0, 2 * x + 1), f(1, 2 * x + 1)));
            } else {
              o[0][x] = to_out2<kB>(f(0, 2 * x), f(0, 2 * x + 1));
              o[1][x] = to_out2<kB>(f(1, 2 * x), f(1, 2 * x + 1));
            }
          }
          // Products beyond fp16's range also go to the workspace in fp32, where
          // the weighted sum finds them: it may be within the range. (Hardly ever:
          // eight instructions per thread and chunk, against twice the bytes of all.)
          if (!kB && a.combine) {
            uint32_t most = 0u;  // the largest magnitudes, in pairs
#pragma unroll
            for (int h = 0; h < 2; ++h)
#pragma unroll
              for (int x = 0; x < 4; ++x) most = max_abs2(most, o[h][x]);
            if (__any_sync(0xffffffffu, (most & 0x7fffu) == kHalfInf || (most >> 16 & 0x7fffu) == kHalfInf)) {
#pragma unroll
              for (int x = 0; x < 8; ++x) {
                const int choice = __shfl_sync(0xffffffffu, chosen, 16 * j + 8 * (x >> 2) + 2 * (lane % 4) + (x & 1));
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                  float* to = p.wide + (size_t)(uint32_t)choice * (uint32_t)width + (s0 + h) * kStripCols + lane / 4 + 8 * (x >> 1 & 1);
                  if (choice >= 0 && s0 + h < limit && fabsf(f(h, x)) >= kHalfInfinite && in_buf(to, p.wide, all + 7, a.err))
                    *to = f(h, x);
                }
              }
            }
          }
          // matrix 2 m + v of a strip: rows 8 m .., columns 8 v ..; a row of the
          // staged chunk has 2 (silu) or 4 pieces of 16 bytes, swizzled by the row
          const int strips_out = a.silu ? 1 : 2;
          const int trow = 8 * (lane / 16) + lane % 8, v = lane / 8 % 2;
          __syncwarp();  // (the chunk before has been read)
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            if (h == strips_out) break;
            const uint32_t piece = a.silu ? (uint32_t)(v ^ (trow >> 2 & 1)) : (uint32_t)((2 * h + v) ^ (trow >> 1 & 3));
            stmatrix_trans(stage0 + (uint32_t)trow * 32u * strips_out + piece * 16u, o[h]);
          }
          __syncwarp();
          // a lane's pieces: silu: row lane / 2, piece lane % 2; else rows lane / 4
          // and 8 + lane / 4, piece lane % 4
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            if (h == strips_out) break;
            const int row = a.silu ? lane / 2 : 8 * h + lane / 4, pc = a.silu ? lane % 2 : lane % 4;
            const uint32_t sw = a.silu ? (uint32_t)(pc ^ (row >> 2 & 1)) : (uint32_t)(pc ^ (row >> 1 & 3));
            const uint4 d = lds128(stage0 + (uint32_t)row * 32u * strips_out + sw * 16u);
            const int f = __shfl_sync(0xffffffffu, chosen, 16 * j + row);
            const int strip = s0 + pc / 2;
            uint16_t* y = reinterpret_cast<uint16_t*>(reinterpret_cast<char*>(out + strip * kStripCols + pc % 2 * 8) +
                                                      (uint64_t)(uint32_t)f * pitch);
            if (f >= 0 && strip < limit && in_buf(y, out, all, a.err)) *reinterpret_cast<uint4*>(y) = d;
          }
        }
      }
      return true;
    };
    bool ok = true;
    int done = 0;  // the tiles whose epilogue this warp has done: [0, done)
    int slot = grp_id;  // the stage's rows' slot
    if (grp_id < total) {
      enter_tile();
      ngrp = group_of(next.kb);
      copy_meta();
    }
    for (int it = 0; grp_id + it * kGroups < total && ok; ++it) {
      if (!(ok = stage(it, slot))) break;
      slot = slot == 0 ? nact - 1 : slot - 1;  // (s + 4) % 5 = (s - 1) % 5
      // the epilogues of the tiles before the converted stage's tile
      const int tile = next.tile;
      for (; ok && done < tile; ++done) ok = epilogue(done);
      if (grp_id + (it + 1) * kGroups < total) {
        next.step(kGroups, nk);
        if (next.tile != tile) enter_tile();
        ngrp = group_of(next.kb);
        copy_meta();
      }
    }
    for (; ok && done < ntl; ++done) ok = epilogue(done);
    copies_wait();
  }

  // the pair's last commit has landed here before the CTA can leave: the last
  // tile's accumulator commit in a normal run (already waited for by the
  // epilogue), the drain commit after an abort
  if (threadIdx.x == 32 * kFirst && ntl > 0) {
    if (*abort_flag == 0) mbar_drain(accum_full(1), (uint32_t)(ntl - 1) & 1u, a.err);
    else mbar_drain(drain_bar, 0, a.err);
  }
  __syncwarp();
  tc_fence_before();
  cluster_sync();  // both CTAs done with the tensor memory and each other's barriers
  if (warp == 1) {
    __syncwarp();
    tc_fence_after();
    pair_tmem_dealloc(tmem_base, 512);
  }
}

// ------------------------------------------------------------------ host

template <bool kB>
cudaError_t launch(const CUtensorMap& tmW, TensorParams p, cudaStream_t stream) {
  const void* kern = reinterpret_cast<const void*>(experts_tc_kernel<kB>);
  cudaError_t e = set_max_smem_once(kern, kSmemBytes);
  if (e != cudaSuccess) return e;
  cudaLaunchConfig_t cfg = {};
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = kSmemBytes;
  cfg.stream = stream;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = 2;
  attr[0].val.clusterDim.y = 1;
  attr[0].val.clusterDim.z = 1;
  attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[1].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;             // the occupancy query takes the cluster shape only
  cfg.gridDim = dim3(2, 1, 1);  // and a grid of whole clusters
  int resident = 0;
  e = max_active_clusters(kern, cfg, &resident);
  if (e != cudaSuccess) return e;
  // persistent: no more clusters than there can be tiles
  const ExpertArgs& a = p.a;
  const long long most = (long long)(choices(a) / (2 * kRows) + (choices(a) < a.E ? choices(a) : a.E)) * p.pairs;
  cfg.gridDim = dim3((unsigned)(2 * (most < resident ? most : resident)), 1, 1);
  cfg.numAttrs = 2;
  return cudaLaunchKernelEx(&cfg, experts_tc_kernel<kB>, tmW, p);
}

}  // namespace

// The products in 16 bits, and in fp32 those that fp16 cannot hold (of both
// types alike: a workspace's size does not depend on the type).
size_t experts_tc_workspace_bytes(int choices, int N, bool combine) {
  return combine ? kWorkspaceFlags + (size_t)choices * N * (sizeof(uint16_t) + sizeof(float)) : 0;
}

cudaError_t launch_experts_tc(ExpertArgs a, bool bf16, void* workspace, cudaStream_t stream) {
  cudaError_t e = device_error_word(&a.err);
  if (e != cudaSuccess) return e;
  CUtensorMap tmW;
  if (!cached_expert_map(&tmW, a.Wq, a.N, a.K, a.E, kAtoms, a.silu)) return cudaErrorInvalidValue;
  const int wide = a.silu ? a.N / 2 : a.N, per = a.silu ? kCols : 2 * kCols;
  TensorParams p = {a, nullptr, nullptr, (wide + per - 1) / per, 1.f / (float)a.group};
  if (a.combine) {
    p.D = reinterpret_cast<uint16_t*>(static_cast<uint8_t*>(workspace) + kWorkspaceFlags);
    p.wide = reinterpret_cast<float*>(p.D + (size_t)choices(a) * a.N);  // (N is a multiple of 16)
  }
  e = bf16 ? launch<true>(tmW, p, stream) : launch<false>(tmW, p, stream);
  return e != cudaSuccess || !a.combine ? e : launch_experts_sum(a, p.D, p.wide, bf16, stream);
}

}  // namespace w4a16
