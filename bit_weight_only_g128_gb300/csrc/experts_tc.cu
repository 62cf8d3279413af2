// W4A16 products grouped by expert on the tensor cores (sm_103a:
// tcgen05.mma.cta_group::2, tensor memory, TMA), for many rows per expert.
//
// Choice f of expert e: Y[f][n] = sum_k A[f or f / top][k] W_e[k][n], with the
// gate/up epilogue silu(gate) * up of columns [gate | up], or the products
// multiplied by their weights and rounded to 16 bits for the sum over a
// token's choices (experts.cu adds them up in fp32).
//
// The contraction is the one of the kernel for one weight (tc_pair.cu): a
// cluster of two CTAs makes a tile of 256 weight columns x up to 192 rows,
// each CTA dequantizing its 128 columns, RNE((q - z) s) in the activations'
// type, straight into tensor memory (the MMA's A operand) and staging half of
// the rows (the B operand). What differs:
//   - An expert's n rows make ceil(n / 192) tiles of the same size, rounded up
//     to 16 rows, and the MMA's N is that size: an expert of 40 rows costs
//     MMAs of 48, not 192. Which tiles there are is known on the device only:
//     every CTA makes the list of the experts' first tiles from the offsets
//     when it starts, and each role walks it (a cluster's tiles ascend).
//   - The rows are gathered by the converting warps: the group that will
//     convert a stage copies the stage's rows two of its stages before
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
//   - K is short (an expert's inner width), so that a tile's end matters: two
//     accumulators of 192 columns take the tiles in turn, and the converting
//     warps store a tile's results 16 rows at a time between the conversions
//     of the next tile's stages, which keeps the MMAs fed meanwhile. The
//     dequantized operand has the remaining 128 columns, four atoms; a stage is
//     one atom.
// Rings, barriers and their invariants are those of tc_pair.cu, without a
// barrier for the rows' arrival. Besides, a
// group finishes a tile's results before it converts a stage of the tile two
// after it, whose accumulator is the same: what a group waits for before a
// stage is the work of earlier stages alone. Every wait is
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
constexpr int kThreads = 64 + 128 * kGroups;
constexpr int kRows = 192;                  // most rows of a tile (MMA N)
constexpr int kMostExperts = 512;
constexpr int kActSlot = kRows / 2 * 128;   // bytes of a CTA's rows of one atom, at most
// the list of tiles in shared memory: offsets and first tiles [E + 1] each
constexpr int kListBytes = ((kMostExperts + 1) * 8 + 127) / 128 * 128;

struct TensorParams {
  ExpertArgs a;
  uint16_t* D;     // combined: [choices][N], the weighted products
  int pairs;       // tiles along the columns
};

// Tile t of the launch (which lies in expert e's): 256 columns (with silu 128
// of gate and of up) x the rows [first, first + n) of the list; size: the
// MMA's N.
struct Tile {
  int e, col, first, n, size;
};

// Ring depths per CTA (a stage is an atom): codes 16 (64 KiB), the rows as
// deep as a group's copies two of its stages ahead need (12 slots of 12 KiB),
// the dequantized operand in the tensor memory that the accumulators leave.
// The invariants of tc_pair.cu: at least as many dequantized slots as groups,
// no more than activation slots, code slots a multiple of the groups.
constexpr int kActSlots = 12, kCodeSlots = 16, kDqSlots = (512 - 2 * kRows) / kAtomCols;
constexpr int kSmemBytes = kActSlots * kActSlot + kCodeSlots * kCodeAtomBytes + 1024 + kBarBytes + kListBytes;
static_assert(kDqSlots >= kGroups && kDqSlots <= kActSlots && kCodeSlots % kGroups == 0 && kSmemBytes <= kSmemLimit &&
                  8 * (kActSlots + kDqSlots + 2 * kCodeSlots + 5) + 8 <= kBarBytes,
              "ring depths break the barriers' invariants");

__device__ __forceinline__ int row_tiles(int n) { return (n + kRows - 1) / kRows; }

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
__device__ __forceinline__ void copies_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
// all but this thread's N most recent groups of copies have landed
template <int N>
__device__ __forceinline__ void copies_wait() { asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory"); }

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
  // of tile i's accumulator, i & 1; phase i >> 1
  auto accum_full = [&](int i) { return bars + 8u * (nact + ndq + 2 * ncode + (i & 1)); };
  auto accum_empty = [&](int i) { return bars + 8u * (nact + ndq + 2 * ncode + 2 + (i & 1)); };  // in the first CTA
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
    const int size = ((n + rt - 1) / rt + 15) & ~15, row = local % rt * size;
    return {e, local / rt, offs[e] + row, min(size, n - row), size};
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
    if (lane == 0 && rank == 0 && total > 0) {
      // ---------------------------------------------------------- MMA issuer (first CTA)
      int slot = 0, w = 0, e = 0;
      uint32_t pw = 0;
      bool ok = mbar_wait_poll(dq_full(0), 0, abort_flag, kErrMma, a.err);
      for (int tl = 0; tl < ntl && ok; ++tl) {
        const uint32_t idesc = f16_idesc(2 * kCols, tile_at(tl, e).size, kB);
        const uint32_t acc = (uint32_t)((tl & 1) * kRows);
        if (tl > 1 && !(ok = mbar_wait_poll(accum_empty(tl), (uint32_t)((tl >> 1) - 1) & 1u, abort_flag, kErrMma, a.err)))
          break;
        const bool more = tl + 1 < ntl;  // another tile's stages follow this tile's last
        for (int kb = 0; kb < nk && ok; ++kb) {
          tc_fence_after();
          const uint32_t bst = base + (uint32_t)slot * kActBytes;
          const uint32_t acol = tmem_base + (uint32_t)(kDqCol0 + w * kAtomCols);
          if (!in_smem(bst, kActBytes, raw, a.err) || !in_tmem((uint32_t)(kDqCol0 + w * kAtomCols), kAtomCols, 512, a.err)) {
            ok = false;
            break;
          }
          const bool next = kb + 1 < nk || more;
          const int w2 = w + 1 == ndq ? 0 : w + 1;
          const uint32_t pw2 = w2 == 0 ? pw ^ 1u : pw;
          bool ready = true;
          const uint64_t bdesc = sw128_kmajor_desc(bst);
#pragma unroll
          for (int kk = 0; kk < kStageK / 16; ++kk) {  // 16 k per MMA: 8 columns of A, 32 bytes of B
            pair_mma_f16_ts(tmem_base + acc, acol + (uint32_t)(8 * kk), bdesc + 2u * kk, idesc, (kb | kk) != 0);
            if (kk == 1 && next) ready = mbar_test(dq_full(w2), pw2);
          }
          pair_commit_both(stage_done(slot));
          slot = slot + 1 == nact ? 0 : slot + 1;
          w = w2;
          pw = pw2;
          if (next && !ready) ok = mbar_wait_poll(dq_full(w), pw, abort_flag, kErrMma, a.err);
        }
        if (ok) pair_commit_both(accum_full(tl));  // the tile's accumulator is complete
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
    const int dw = warp - 2;
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
        for (int n = threadIdx.x - 64; f >= 0 && n < width; n += 128 * kGroups) {
          uint16_t* y = a.Y + (size_t)f * width + n;
          if (in_buf(y, a.Y, (size_t)choices(a) * width, a.err)) *y = 0;
        }
      }

    // the strip of this lane in a tile, of all experts' strips; -1: beyond the columns
    auto strip_of = [&](const Tile& t) {
      const int s = first_strip(t) + (a.silu ? q : ls);
      return s < limit ? t.e * strips + s + (a.silu && lane >= 16 ? limit : 0) : -1;
    };
    // scale and zero point of this column for a stage, in order, kGroups stages
    // apart (taken apart where they are used: their loads are in flight until then)
    int mi = grp_id, me = 0;
    SeqPos mseq{grp_id, 0};
    mseq.step(0, nk);
    int mstrip = mi < total ? strip_of(tile_at(mseq.tile, me)) : -1;
    int mgrp = mseq.kb * kStageK / a.group;
    int mgend = (mgrp + 1) * a.group;
    struct Meta {
      uint16_t s;  // scale bits
      uint8_t z;   // the zero points of columns cp and cp + 8
    };
    auto load_meta = [&]() -> Meta {
      Meta v = {0, 0};
      if (mi < total && mstrip >= 0) {
        const size_t pg = (size_t)mstrip * G + mgrp;
        const uint8_t* zp = reinterpret_cast<const uint8_t*>(a.Zp);
        v.s = __ldg(ld_at(a.Sp + pg * 16 + 2 * cp + (hi ? 1 : 0), a.Sp, (size_t)G * a.N * a.E, a.err));
        v.z = __ldg(ld_at(zp + pg * 8 + cp, zp, (size_t)G * a.N / 2 * a.E, a.err));
      }
      mi += kGroups;
      const int tl = mseq.tile;
      mseq.step(kGroups, nk);
      if (mseq.tile != tl) {
        if (mi < total) mstrip = strip_of(tile_at(mseq.tile, me));
        mgrp = 0;
        mgend = a.group;
      }
      while (mseq.kb * kStageK >= mgend) {
        ++mgrp;
        mgend += a.group;
      }
      return v;
    };
    const uint32_t dq_remote0 = cluster_addr(dq_full(0), 0);     // the first CTA's dq_full(0)
    const uint32_t empty_remote = cluster_addr(accum_empty(0), 0);  // the first CTA's accum_empty(0)
    // a wait that every lane of the warp passes or every lane gives up on:
    // the tensor-memory stores and loads that follow are .sync.aligned
    auto warp_wait = [&](uint32_t bar, uint32_t parity, bool poll, int code) -> bool {
      const bool ok = poll ? mbar_wait_poll(bar, parity, abort_flag, code, a.err)
                           : mbar_wait(bar, parity, abort_flag, code, a.err);
      return __all_sync(0xffffffffu, ok);
    };
    // the rows of the group's stages: this warp copies those of steps q, q + 4,
    // ... (step i: rows 4 i .. 4 i + 3 of this CTA's half), this lane the 16
    // bytes lane % 8 of row 4 i + lane / 8. aseq: the next stage to copy.
    constexpr int kSteps = kRows / 2 / 16;
    int rows[kSteps];  // in A
    int ai = grp_id, ae = 0, ahalf = 0;
    SeqPos aseq{grp_id, 0};
    aseq.step(0, nk);
    RingPos apos;
    apos.init(grp_id, nact);
    const size_t a_all = a_elements(a) - 7;
    // chunk lane % 8 of row lane / 8 of a step, swizzled by the row's number in
    // its group of eight: 4 (i & 1) + lane / 8, and i is as odd as q
    const uint32_t place = (uint32_t)q * 512u + (uint32_t)(lane / 8) * 128u +
                           (uint32_t)((lane % 8) ^ (lane / 8 + 4 * (q & 1))) * 16u;
    auto load_rows = [&]() {
      const Tile t = tile_at(aseq.tile, ae);
      ahalf = t.size / 2;
#pragma unroll
      for (int j = 0; j < kSteps; ++j) {
        const int i = 4 * (q + 4 * j) + lane / 8;
        if (i < ahalf) {
          const int f = choice_of(a, t.first + min((int)rank * ahalf + i, t.n - 1));
          rows[j] = f < 0 ? 0 : a.per_choice ? f : f / a.top;
        }
      }
    };
    auto copy_rows = [&]() {
      if (ai < total) {
        const uint32_t to = base + (uint32_t)apos.slot * kActBytes + place;
        const uint16_t* from = a.A + aseq.kb * kStageK + lane % 8 * 8;
#pragma unroll
        for (int j = 0; j < kSteps; ++j)
          if (4 * (q + 4 * j) < ahalf && in_smem(to + 2048u * j, 16, raw, a.err))
            copy16(to + 2048u * j, ld_at(from + (size_t)rows[j] * a.K, a.A, a_all, a.err));
        ai += kGroups;
        apos.step(kGroups, nact);
        const int tl = aseq.tile;
        aseq.step(kGroups, nk);
        if (aseq.tile != tl && ai < total) load_rows();
      }
      copies_commit();
    };
    constexpr int kAhead = nact - ndq;  // stages: the slot of stage s + kAhead was that of stage s - ndq
    static_assert(kAhead == 2 * kGroups, "two groups of copies are in flight beside a stage's own");
    if (ai < total) load_rows();
    copy_rows();
    copy_rows();
    RingPos spos_code, spos_act;
    spos_code.init(grp_id, ncode);
    spos_act.init(grp_id, nact);
    int sw = grp_id % ndq;
    SeqPos sseq{grp_id, 0};
    sseq.step(0, nk);
    int stile = 0;  // the tile of the stage converted last
    auto stage = [&](int s, const Meta& meta) -> bool {
      const int cs = spos_code.slot, w = sw;
      const uint32_t code_par = spos_code.phase;
      const RingPos prev = spos_act.before(ndq, nact);  // stage s - dq_slots (dq_slots <= act_slots)
      stile = sseq.tile;
      spos_code.step(kGroups, ncode);
      spos_act.step(kGroups, nact);
      sw += kGroups;
      while (sw >= ndq) sw -= ndq;
      sseq.step(kGroups, nk);
      if (!warp_wait(code_full(cs), code_par, false, kErrDequant)) return false;
      const uint32_t cb = code_base + (uint32_t)cs * kCodeBytes;
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
      if (lane == 0) mbar_arrive(code_empty(cs));  // the codes are in registers
      const uint32_t z = ((uint32_t)meta.z >> (hi ? 4 : 0)) & 15u;
      const uint16_t sc = meta.s;
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
      // (the slot is waited for with the cells in registers: what is between its
      // last MMA and its next is then the store alone)
      if (s >= ndq) {
        if (!warp_wait(stage_done(prev.slot), prev.phase, true, kErrDequant)) return false;
        tc_fence_after();
      }
      copy_rows();  // of stage s + kAhead, to the slot of the stage waited for
      if (in_tmem((uint32_t)(kDqCol0 + w * kAtomCols), kAtomCols, 512, a.err))
        tmem_st32(tmem_base + tlane + (uint32_t)(kDqCol0 + w * kAtomCols), r);
      tmem_wait_st();
      // this warp's rows of the stage have landed (the MMAs read them too)
      copies_wait<2>();
      fence_async_shared();  // (the copies wrote them through the generic proxy)
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive_remote(dq_remote0 + 8u * w);
      return true;
    };
    // the epilogue of this warp: tensor-memory lanes 32q..32q+31 are this CTA's
    // columns, an accumulator's columns the tile's rows, 16 at a time by the
    // groups in turn. done: the tiles that the warp has finished; of the next
    // one, et and the group's next chunk of 16 rows, of which lane l (and 16 +
    // l) holds row l's choice and weight.
    int done = 0, ee = 0, chunk = 0, of = -1;
    float factor = 1.f;
    Tile et{};
    auto load_chunk = [&]() {
      const int r = 16 * chunk + (lane & 15);
      of = r < et.n ? choice_of(a, et.first + r) : -1;
      if (a.combine) factor = of >= 0 ? *ld_at(a.weights + of, a.weights, (size_t)choices(a), a.err) : 1.f;
    };
    auto begin_tile = [&]() {
      if (done >= ntl) return;
      et = tile_at(done, ee);
      chunk = grp_id;
      load_chunk();
    };
    // the tile's next chunk; the tile's accumulator is complete
    uint16_t* out = a.combine ? p.D : a.Y;
    const size_t all = (size_t)choices(a) * width;
    auto store_chunk = [&]() {
      if (16 * chunk < et.n) {
        const uint32_t col = (uint32_t)((done & 1) * kRows + 16 * chunk);
        const int s = first_strip(et) + (a.silu ? q : ls);
        const bool live = s < limit;
        uint16_t* to = out + s * kStripCols + c;
        uint32_t r[16];
        tc_fence_after();
        if (in_tmem(col, 16, kDqCol0, a.err)) tmem_ld16(tmem_base + tlane + col, r);
        tmem_wait_ld();
        if (a.silu) {
          // lanes 0..15 finish rows 0..7 of the chunk, lanes 16..31 rows 8..15
#pragma unroll
          for (int k = 0; k < 8; ++k) {
            const uint32_t other = __shfl_xor_sync(0xffffffffu, lane < 16 ? r[k + 8] : r[k], 16);
            const float g = __uint_as_float(lane < 16 ? r[k] : other);
            const float u = __uint_as_float(lane < 16 ? other : r[k + 8]);
            const int f = __shfl_sync(0xffffffffu, of, k + (lane < 16 ? 0 : 8));
            uint16_t* y = to + (size_t)f * width;
            if (f >= 0 && live && in_buf(y, out, all, a.err)) *y = to_out<kB>(silu_times(g, u));
          }
        } else {
#pragma unroll
          for (int k = 0; k < 16; ++k) {
            const int f = __shfl_sync(0xffffffffu, of, k);
            const float w = a.combine ? __shfl_sync(0xffffffffu, factor, k) : 1.f;
            uint16_t* y = to + (size_t)f * width;
            if (f >= 0 && live && in_buf(y, out, all, a.err)) *y = to_out<kB>(__uint_as_float(r[k]) * w);
          }
        }
      }
      chunk += kGroups;
      if (16 * chunk < et.n) {
        load_chunk();
      } else {  // the warp has read all it reads of this accumulator
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive_remote(empty_remote + 8u * (done & 1));
        ++done;
        begin_tile();
      }
    };
    auto wait_tile = [&]() { return warp_wait(accum_full(done), (uint32_t)(done >> 1) & 1u, true, kErrEpilogue); };
    // scales and zero points, loaded two of this group's stages before their own
    Meta m0s = load_meta(), m1s = load_meta();
    begin_tile();
    bool ok = true;
    for (int s = grp_id; s < total && ok; s += kGroups) {
      const Meta m2s = load_meta();  // stage s + 2 groups
      while (ok && done + 1 < sseq.tile)
        if ((ok = wait_tile())) store_chunk();
      if (ok) ok = stage(s, m0s);
      // a chunk of an earlier tile, if its accumulator is complete
      if (ok && done < stile &&
          __all_sync(0xffffffffu, mbar_test(accum_full(done), (uint32_t)(done >> 1) & 1u)))
        store_chunk();
      m0s = m1s;
      m1s = m2s;
    }
    while (ok && done < ntl)
      if ((ok = wait_tile())) store_chunk();
    copies_wait<0>();
  }

  // the pair's last commit has landed here before the CTA can leave: the last
  // tile's accumulator commit in a normal run (already waited for by the
  // epilogue), the drain commit after an abort
  if (threadIdx.x == 64 && ntl > 0) {
    if (*abort_flag == 0) mbar_drain(accum_full(ntl - 1), (uint32_t)((ntl - 1) >> 1) & 1u, a.err);
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
  const long long most = (long long)(choices(a) / kRows + (choices(a) < a.E ? choices(a) : a.E)) * p.pairs;
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
