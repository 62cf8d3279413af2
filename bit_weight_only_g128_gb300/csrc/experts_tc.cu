// W4A16 products grouped by expert on the tensor cores (sm_103a:
// tcgen05.mma.cta_group::2, tensor memory, TMA), for many rows per expert.
//
// Choice f of expert e: Y[f][n] = sum_k A[f or f / top][k] W_e[k][n], with the
// gate/up epilogue silu(gate) * up of columns [gate | up], or the products
// multiplied by their weights and rounded to 16 bits for the sum over a
// token's choices (experts.cu adds them up in fp32).
//
// The contraction is the one of the kernel for one weight (tc_pair.cu): a
// cluster of two CTAs makes a tile of 256 weight columns, each CTA dequantizing
// its 128 columns, RNE((q - z) s) in the activations' type, straight into
// tensor memory (the MMA's A operand) and staging half of the rows (the B
// operand). What differs:
//   - A tile has up to 384 rows in two parts of up to 192, each with its own
//     accumulator: a dequantized atom serves both, so that conversions, whose
//     instructions bound the kernel below that, take half as many per row.
//     An expert's n rows make ceil(n / 384) tiles of the same size, and the
//     MMA's N is a part's size, rounded up to 16: an expert of 40 rows costs
//     MMAs of 48. Which tiles there are is known on the device only: every CTA
//     makes the list of the experts' first tiles from the offsets when it
//     starts, and each role walks it (a cluster's tiles ascend).
//   - The rows are gathered by the converting warps: the group that will
//     convert a stage copies the stage's rows one of its stages before
//     (cp.async, eight lanes a row of 128 bytes, to the swizzled places), and
//     each of its warps waits for its own copies before it arrives for the
//     stage. (tile::gather4 copies by the lanes of one warp took about 95
//     cycles each, one warp's cp.async about 85: the MMAs waited for rows most
//     of the time.) Places beyond a tile's rows repeat its last row; their
//     results are not stored.
//   - With silu(gate) * up a CTA's eight strips are four of gate columns and
//     the four of up columns beside them (one 4-D copy), placed so that a
//     warp's lanes 0..15 hold gate and 16..31 up of the same 16 results: one
//     shuffle per two results brings them together in fp32, and the output is
//     half as wide.
//   - K is short (an expert's inner width), so that a tile's end matters: the
//     converting warps take a part's accumulator to registers, hand it back
//     and only then convert and store, one part after the other. The next
//     tile begins with the first part's MMAs of the stages that are converted
//     already, and catches up with the second part's when its accumulator is
//     free.
// Rings, barriers and their invariants are those of tc_pair.cu, without a
// barrier for the rows' arrival. A stage is one atom. Every wait is
// bounded; a wait that gives up sets the library's error word, and its CTA
// drains and leaves through the same final cluster barrier as a normal run.
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
constexpr int kRows = 192;                  // most rows of a part (MMA N); a tile has two
constexpr int kMostExperts = 512;
constexpr int kPartSlot = kRows / 2 * 128;  // bytes of a CTA's rows of one atom of a part, at most
constexpr int kActSlot = 2 * kPartSlot;
// the list of tiles in shared memory: offsets and first tiles [E + 1] each
constexpr int kListBytes = ((kMostExperts + 1) * 8 + 127) / 128 * 128;

struct TensorParams {
  ExpertArgs a;
  uint16_t* D;     // combined: [choices][N], the weighted products
  int pairs;       // tiles along the columns
};

// Tile t of the launch (which lies in expert e's): 256 columns (with silu 128
// of gate and of up) x the rows [first, first + n) of the list, in `parts` parts
// of `size` (the MMA's N).
struct Tile {
  int e, col, first, n, parts, size;
};

// Ring depths per CTA (a stage is an atom): the dequantized operand in the
// tensor memory beside the accumulators, four slots; the rows four stages
// deeper, which is how far ahead a group copies them (8 slots of 24 KiB); codes
// four. The invariants of tc_pair.cu: at least as many dequantized slots as
// groups, no more than activation slots, code slots a multiple of the groups.
constexpr int kActSlots = 8, kCodeSlots = 4, kDqSlots = (512 - 2 * kRows) / kAtomCols;
constexpr int kMetaBytes = 128 * kGroups * 8;  // scales and zero points of a stage of every converting thread
constexpr int kSmemBytes = kActSlots * kActSlot + kCodeSlots * kCodeAtomBytes + 1024 + kBarBytes + kListBytes + 2 * kMetaBytes;
static_assert(kDqSlots >= kGroups && kDqSlots <= kActSlots && kCodeSlots % kGroups == 0 && kSmemBytes <= kSmemLimit &&
                  8 * (kActSlots + kDqSlots + 2 * kCodeSlots + 5) + 8 <= kBarBytes,
              "ring depths break the barriers' invariants");

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

__device__ __forceinline__ void copy16(uint32_t to, const void* from) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(to), "l"(from) : "memory");
}
__device__ __forceinline__ void copy4(uint32_t to, const void* from) {
  asm volatile("cp.async.ca.shared.global [%0], [%1], 4;" ::"r"(to), "l"(from) : "memory");
}
// One lane of a converged warp.
__device__ __forceinline__ bool elect_one() {
  uint32_t ok;
  asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.u32 %0, 1, 0, p;\n\t}" : "=r"(ok));
  return ok != 0;
}
// all of this thread's copies have landed
__device__ __forceinline__ void copies_wait() { asm volatile("cp.async.wait_all;" ::: "memory"); }

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
  constexpr uint32_t kActBytes = kActSlot, kCodeBytes = kCodeAtomBytes;
  constexpr int kDqCol0 = 2 * kRows;  // tensor memory: two accumulators, then the dequantized operand
  // [activation ring | code ring | barriers | list of tiles], 1024-aligned slots
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
  volatile int* abort_flag = reinterpret_cast<volatile int*>(gen_base + (tmem_slot + 4u - base));
  int* offs = reinterpret_cast<int*>(gen_base + (bars + kBarBytes - base));  // [E + 1]
  int* firsts = offs + kMostExperts + 1;                                     // [E + 1]: an expert's first tile

  const uint32_t rank = cluster_rank();  // 0: the CTA that issues the MMAs
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int cluster = blockIdx.x >> 1, clusters = gridDim.x >> 1;
  const int nk = a.K / kStageK;  // stages of one tile

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
    const int n = offs[e + 1] - offs[e], rt = row_tiles(n), local = t - firsts[e];
    const int each = (n + rt - 1) / rt, parts = each > kRows ? 2 : 1;
    const int size = ((each + parts - 1) / parts + 15) & ~15, row = local % rt * parts * size;
    return {e, local / rt, offs[e] + row, min(parts * size, n - row), parts, size};
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
          tma_load_4d(to, &tmW, 0, seq.kb * 4, first_strip(t), a.silu ? 2 * t.e : t.e, code_full(pos.slot));
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
      // stage n of the sequence has activation slot n & 7 and dequantized slot n & 3
      static_assert(nact == 8 && ndq == 4, "slots by the stage's number alone");
      const uint64_t bdesc0 = sw128_kmajor_desc(base);
      int n = 0;
      int e = 0;
      bool ok = true;
      for (int tl = 0; tl < ntl && ok; ++tl) {
        const Tile t = tile_at(tl, e);
        const uint32_t idesc = f16_idesc(2 * kCols, t.size, kB);
        const uint32_t phase = (uint32_t)(tl - 1) & 1u;  // of the accumulators' release by the tile before
        auto ready = [&](int i) {
          return mbar_wait_poll(dq_full(i & 3), (uint32_t)(i >> 2) & 1u, abort_flag, kErrMma, a.err);
        };
        // the four MMAs (16 k: 8 columns of A, 32 bytes of B) of a part of a stage
        auto mmas = [&](int i, int part, bool first) {
          const uint32_t place = (uint32_t)((i & 7) * kActSlot + part * kPartSlot);
          const uint32_t acol = (uint32_t)(kDqCol0 + (i & 3) * kAtomCols);
          if (!in_smem(base + place, kPartSlot, raw, a.err) || !in_tmem(acol, kAtomCols, 512, a.err)) return;
          const uint64_t bdesc = bdesc0 + (place >> 4);
#pragma unroll
          for (int kk = 0; kk < kStageK / 16; ++kk)
            pair_mma_f16_ts(tmem_base + (uint32_t)(part * kRows), tmem_base + acol + (uint32_t)(8 * kk), bdesc + 2u * kk,
                            idesc, !first || kk != 0);
        };
        if (tl > 0 && !(ok = mbar_wait_poll(accum_empty(0), phase, abort_flag, kErrMma, a.err))) break;
        // after another tile, the first part of the stages that there are slots
        // for, then the second (no slot is freed in between)
        const int begin = tl > 0 && t.parts == 2 ? min(nk, ndq) : 0;
        for (int kb = 0; kb < begin && ok; ++kb) {
          if (!(ok = ready(n + kb))) break;
          tc_fence_after();
          mmas(n + kb, 0, kb == 0);
        }
        if (ok && begin == nk) pair_commit_both(accum_full(0));
        if (ok && tl > 0) ok = mbar_wait_poll(accum_empty(1), phase, abort_flag, kErrMma, a.err);
        for (int kb = 0; kb < begin && ok; ++kb, ++n) {
          mmas(n, 1, kb == 0);
          pair_commit_both(stage_done(n & 7));
        }
        for (int kb = begin; kb < nk && ok; ++kb, ++n) {
          if (!(ok = ready(n))) break;
          tc_fence_after();
          mmas(n, 0, kb == 0);
          if (kb + 1 == nk) pair_commit_both(accum_full(0));
          if (t.parts == 2) mmas(n, 1, kb == 0);
          pair_commit_both(stage_done(n & 7));
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
    const uint32_t empty_remote = cluster_addr(accum_empty(0), 0);     // the first CTA's accum_empty(0)
    // a wait that every lane of the warp passes or every lane gives up on:
    // the tensor-memory stores and loads that follow are .sync.aligned
    auto warp_wait = [&](uint32_t bar, uint32_t parity, bool poll, int code) -> bool {
      const bool ok = poll ? mbar_wait_poll(bar, parity, abort_flag, code, a.err)
                           : mbar_wait(bar, parity, abort_flag, code, a.err);
      return __all_sync(0xffffffffu, ok);
    };

    // The group's stages are grp_id, grp_id + 4, ...: its it-th stage has the
    // code slot and the dequantized slot grp_id, and the activation slots
    // grp_id and grp_id + 4 in turn. `next` is the stage whose rows and scales
    // are fetched while the one before it is converted: its place, its tile's
    // expert, this lane's strip of all experts' strips (-1: beyond the
    // columns), the group of its scale and the k where the group after it
    // starts, and the rows.
    static_assert(ncode == kGroups && ndq == kGroups && nact == 2 * kGroups, "slots by the group's number alone");
    SeqPos next{grp_id, 0};
    next.step(0, nk);
    int ne = 0, nstrip = -1, ngrp = next.kb * kStageK / a.group, ngend = (ngrp + 1) * a.group;
    // Rows: of each part this warp copies those of steps q, q + 4, ... (step
    // i: rows 4 i .. 4 i + 3 of this CTA's half of it), a lane the 16 bytes lane
    // % 8 of row lane / 8 of each; lane 4 j + r holds which row of A is the
    // r-th of the warp's j-th step, held[part].
    constexpr int kSteps = kRows / 2 / 16;
    static_assert(4 * kSteps <= 32, "a row per lane");
    int held[2] = {0, 0}, half = 0;  // half: of a part's rows; minus that with one part
    auto enter_tile = [&]() {
      const Tile t = tile_at(next.tile, ne);
      const int st = first_strip(t) + (a.silu ? q : ls);
      nstrip = st < limit ? t.e * strips + st + (a.silu && lane >= 16 ? limit : 0) : -1;
      half = t.size / 2;
      const int i = 4 * (q + lane / 4 * 4) + lane % 4;
#pragma unroll
      for (int part = 0; part < 2; ++part) {
        if (part == t.parts) break;
        const int f = choice_of(a, t.first + min(part * t.size + (int)rank * half + min(i, half - 1), t.n - 1));
        held[part] = f < 0 ? 0 : a.per_choice ? f : f / a.top;
      }
      if (t.parts == 1) half = -half;
    };
    // the lane's scale and zero point words of a stage, in shared memory by the
    // stage's parity: scales of columns cp and cp + 8, and zero points of columns
    // cp & 4 .. (cp & 4) + 3, each with its column + 8
    const uint32_t meta0 = bars + kBarBytes + kListBytes + (uint32_t)(dw * 32 + lane) * 8u;
    auto copy_meta = [&](int it) {
      if (nstrip < 0) return;
      const size_t pg = (size_t)nstrip * G + ngrp;
      const uint32_t* sp = reinterpret_cast<const uint32_t*>(a.Sp);
      const uint32_t to = meta0 + (uint32_t)(it & 1) * kMetaBytes;
      copy4(to, ld_at(sp + pg * 8 + cp, sp, (size_t)G * a.N * a.E / 2, a.err));
      copy4(to + 4, ld_at(a.Zp + pg * 2 + cp / 4, a.Zp, (size_t)G * a.N * a.E / 8, a.err));
    };
    // chunk lane % 8 of row lane / 8 of a step, swizzled by the row's number in
    // its group of eight: 4 (i & 1) + lane / 8, and i is as odd as q
    const uint32_t place = (uint32_t)q * 512u + (uint32_t)(lane / 8) * 128u +
                           (uint32_t)((lane % 8) ^ (lane / 8 + 4 * (q & 1))) * 16u;
    auto copy_rows = [&](int it) {  // of the group's it-th stage
      const uint32_t to = base + (uint32_t)(grp_id + (it & 1) * kGroups) * kActBytes + place;
      const char* from = reinterpret_cast<const char*>(a.A + next.kb * kStageK + lane % 8 * 8);
      const uint32_t pitch = 2u * (uint32_t)a.K;  // bytes of a row
      const int rows = abs(half);
#pragma unroll
      for (int part = 0; part < 2; ++part) {
        if (part == 1 && half < 0) break;
        uint32_t row[kSteps];
#pragma unroll
        for (int j = 0; j < kSteps; ++j) row[j] = (uint32_t)__shfl_sync(0xffffffffu, held[part], 4 * j + lane / 8);
#pragma unroll
        for (int j = 0; j < kSteps; ++j) {
          const uint32_t dst = to + (uint32_t)part * kPartSlot + 2048u * j;
          const uint16_t* src = reinterpret_cast<const uint16_t*>(from + (uint64_t)row[j] * pitch);
          if (4 * (q + 4 * j) < rows && in_smem(dst, 16, raw, a.err))
            copy16(dst, ld_at(src, a.A, a_elements(a) - 7, a.err));
        }
      }
    };
    // converts the group's it-th stage and copies the rows of the one after it
    auto stage = [&](int it, bool more) -> bool {
      // this warp's rows of the stage (the MMAs read them too), and its scales
      copies_wait();
      fence_async_shared();  // (the copies wrote them through the generic proxy)
      uint32_t mscale, mzero;
      asm volatile("ld.shared.v2.u32 {%0, %1}, [%2];" : "=r"(mscale), "=r"(mzero) : "r"(meta0 + (uint32_t)(it & 1) * kMetaBytes) : "memory");
      if (!warp_wait(code_full(grp_id), (uint32_t)it & 1u, false, kErrDequant)) return false;
      const uint32_t cb = code_base + (uint32_t)grp_id * kCodeBytes;
      uint32_t wl[4], wh[4];  // k-octets l and 4 + l
      const uint32_t row = (uint32_t)(ls * 4 + (cp >> 1));  // 128-byte row of the tile
#pragma unroll
      for (int l = 0; l < 4; ++l) {
        const uint32_t chunk = ((uint32_t)(4 * (cp & 1) + l)) ^ (row & 7u);  // 128-byte swizzle
        const uint32_t at = cb + row * 128u + (chunk << 4);
        const uint4 v = lds128(in_smem(at, 16, raw, a.err) ? at : cb);
        wl[l] = hi ? v.y : v.x;
        wh[l] = hi ? v.w : v.z;
      }
      __syncwarp();
      if (lane == 0) mbar_arrive(code_empty(grp_id));  // the codes are in registers
      const uint32_t z = (mzero >> (8 * (cp & 3) + (hi ? 4 : 0))) & 15u;
      const uint16_t sc = (uint16_t)(mscale >> (hi ? 16 : 0));
      uint32_t r[32];  // cell j = (deq[2j], deq[2j + 1]): k-octet o fills cells 4o..4o+3
#pragma unroll
      for (int l = 0; l < 4; ++l) {
        uint32_t o0[4], o1[4];
        if (kB) {
          const DeqConstBf16 dc = make_deq_const_bf16(z, sc);
          dequant_word_bf16(wl[l], dc, o0);
          dequant_word_bf16(wh[l], dc, o1);
        } else {
          const DeqConst dc = make_deq_const(z, sc);
          dequant_word(wl[l], dc, o0);
          dequant_word(wh[l], dc, o1);
        }
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          r[4 * l + j] = o0[j];
          r[16 + 4 * l + j] = o1[j];
        }
      }
      // the slot's MMAs, of the group's stage before, are done (waited for with
      // the cells in registers: what is between them and the slot's next MMAs is
      // then the store alone)
      if (it > 0) {
        if (!warp_wait(stage_done(grp_id + ((it - 1) & 1) * kGroups), (uint32_t)((it - 1) >> 1) & 1u, true, kErrDequant))
          return false;
        tc_fence_after();
      }
      const uint32_t col = (uint32_t)(kDqCol0 + grp_id * kAtomCols);
      if (in_tmem(col, kAtomCols, 512, a.err)) tmem_st32(tmem_base + tlane + col, r);
      tmem_wait_st();
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive_remote(dq_remote);
      if (more) {  // the stage after it, to the slot of the stage waited for
        copy_meta(it + 1);
        copy_rows(it + 1);
      }
      return true;
    };
    // this warp's part of tile i's epilogue: tensor-memory lanes 32q..32q+31
    // are this CTA's columns, an accumulator's columns the rows of a part, 16
    // at a time by the groups in turn
    constexpr int kChunks = kRows / 16 / kGroups;
    int ee = 0;
    uint16_t* out = a.combine ? p.D : a.Y;
    const size_t all = (size_t)choices(a) * width - 1;
    auto epilogue = [&](int i) -> bool {
      const Tile t = tile_at(i, ee);
      const int s = first_strip(t) + (a.silu ? q : ls);
      const bool live = s < limit;
      // two neighbouring columns at a time: even lanes finish one row, odd
      // lanes the next, of which each gives the other its own column
      char* to = reinterpret_cast<char*>(out + s * kStripCols + (c & ~1));
      const bool odd = lane & 1;
      // the choices of the warp's chunks and their weights, on their way while
      // it waits: lane l holds row l of a part's first (0) and third (1) chunk,
      // lane 16 + l that of the second
      int of[2][2];
      float factor[2][2];
#pragma unroll
      for (int part = 0; part < 2; ++part)
#pragma unroll
        for (int m = 0; m < 2; ++m) {
          const int k = 16 * (grp_id + (2 * m + lane / 16) * kGroups) + lane % 16;
          of[part][m] = k < t.size && part * t.size + k < t.n && part < t.parts ? choice_of(a, t.first + part * t.size + k) : -1;
        }
#pragma unroll
      for (int part = 0; part < 2; ++part)
#pragma unroll
        for (int m = 0; m < 2; ++m)
          factor[part][m] =
              a.combine && of[part][m] >= 0 ? *ld_at(a.weights + of[part][m], a.weights, (size_t)choices(a), a.err) : 1.f;
      static_assert(kChunks <= 4, "two registers of rows");
      for (int part = 0; part < 2; ++part) {
        const int n = part < t.parts ? min(t.size, t.n - part * t.size) : 0;
        if (!warp_wait(accum_full(part), (uint32_t)i & 1u, true, kErrEpilogue)) return false;
        tc_fence_after();
#pragma unroll 1
        for (int j = 0; j < kChunks; ++j) {
          const int row0 = 16 * (grp_id + j * kGroups);
          uint32_t r[16];
          const uint32_t col = (uint32_t)(part * kRows + row0);
          if (row0 < n && in_tmem(col, 16, kDqCol0, a.err)) tmem_ld16(tmem_base + tlane + col, r);
          tmem_wait_ld();
          if (j + 1 == kChunks) {
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive_remote(empty_remote + 8u * part);
          }
          if (row0 >= n) continue;
          const int chosen = part ? (j > 1 ? of[1][1] : of[1][0]) : (j > 1 ? of[0][1] : of[0][0]);
          const float weight = part ? (j > 1 ? factor[1][1] : factor[1][0]) : (j > 1 ? factor[0][1] : factor[0][0]);
          auto store = [&](int row, float lo, float hi) {
            const int f = __shfl_sync(0xffffffffu, chosen, row + j % 2 * 16);
            if (a.combine) {
              const float w = __shfl_sync(0xffffffffu, weight, row + j % 2 * 16);
              lo *= w, hi *= w;
            }
            uint16_t* y = reinterpret_cast<uint16_t*>(to + (uint64_t)(uint32_t)f * (2u * (uint32_t)width));
            if (f >= 0 && live && in_buf(y, out, all, a.err)) *reinterpret_cast<uint32_t*>(y) = to_out2<kB>(lo, hi);
          };
          if (a.silu) {
            // lanes 0..15 finish rows 0..7 of the chunk, lanes 16..31 rows 8..15
#pragma unroll
            for (int k = 0; k < 8; k += 2) {
              float v[2];
#pragma unroll
              for (int h = 0; h < 2; ++h) {
                const uint32_t other = __shfl_xor_sync(0xffffffffu, lane < 16 ? r[k + h + 8] : r[k + h], 16);
                const float g = __uint_as_float(lane < 16 ? r[k + h] : other);
                const float u = __uint_as_float(lane < 16 ? other : r[k + h + 8]);
                v[h] = silu_times(g, u);
              }
              const float other = __shfl_xor_sync(0xffffffffu, odd ? v[0] : v[1], 1);
              store(k + (odd ? 1 : 0) + (lane < 16 ? 0 : 8), odd ? other : v[0], odd ? v[1] : other);
            }
          } else {
#pragma unroll
            for (int k = 0; k < 16; k += 2) {
              const float v0 = __uint_as_float(r[k]), v1 = __uint_as_float(r[k + 1]);
              const float other = __shfl_xor_sync(0xffffffffu, odd ? v0 : v1, 1);
              store(k + (odd ? 1 : 0), odd ? other : v0, odd ? v1 : other);
            }
          }
        }
      }
      return true;
    };
    bool ok = true;
    int done = 0;  // the tiles whose epilogue this warp has done: [0, done)
    if (grp_id < total) {
      enter_tile();
      copy_meta(0);
      copy_rows(0);
    }
    for (int s = grp_id, it = 0; s < total && ok; s += kGroups, ++it) {
      const int tile = next.tile;
      const bool more = s + kGroups < total;
      next.step(kGroups, nk);
      if (more && next.tile != tile) {
        enter_tile();
        ngrp = 0;
        ngend = a.group;
      }
      while (next.kb * kStageK >= ngend) {
        ++ngrp;
        ngend += a.group;
      }
      ok = stage(it, more);
      // the epilogues of the tiles before the converted stage's tile
      for (; ok && done < tile; ++done) ok = epilogue(done);
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
  cudaError_t e = set_max_smem_once(kern, kSmemLimit);
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

size_t experts_tc_workspace_bytes(int choices, int N, bool combine) {
  return combine ? kWorkspaceFlags + (size_t)choices * N * sizeof(uint16_t) : 0;
}

cudaError_t launch_experts_tc(ExpertArgs a, bool bf16, void* workspace, cudaStream_t stream) {
  cudaError_t e = device_error_word(&a.err);
  if (e != cudaSuccess) return e;
  CUtensorMap tmW;
  if (!cached_expert_map(&tmW, a.Wq, a.N, a.K, a.E, 1, a.silu)) return cudaErrorInvalidValue;
  const int wide = a.silu ? a.N / 2 : a.N, per = a.silu ? kCols : 2 * kCols;
  TensorParams p = {a, workspace ? reinterpret_cast<uint16_t*>(static_cast<uint8_t*>(workspace) + kWorkspaceFlags) : nullptr,
                    (wide + per - 1) / per};
  e = bf16 ? launch<true>(tmW, p, stream) : launch<false>(tmW, p, stream);
  return e != cudaSuccess || !a.combine ? e : launch_experts_sum(a, p.D, bf16, stream);
}

}  // namespace w4a16
