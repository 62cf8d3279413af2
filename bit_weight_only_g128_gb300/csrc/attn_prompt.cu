// Causal attention of prompts over the paged cache on the tensor cores.
//
// For the rows of a sequence (a row is a query token and one of the G =
// heads / kv_heads query heads of a key/value head; rows of one token are
// adjacent, so that they share the keys' tiles) and tiles of 128 keys:
//   S = Q K^T, x = S scale log2 e (-inf where the row may not see the key),
//   P = 2^(x - m), l += row sums of P, O += P V; at the end O / l.
// m is a running maximum that follows the row's true maximum only when that
// is more than 2^8 above it: P stays within 2^8 (fp16 holds it, the sums are
// fp32) and O is rarely rescaled.
//
// Bound: the tensor cores, 4 D operations per row and key. One block per SM
// takes units of 256 rows from a queue (the most keys of a sequence first),
// two tiles of 128 whose softmax and products alternate: while one tile's 128
// threads (a row each) form P, the tensor cores work on the other tile. Every
// role runs through the units by itself, so that a unit's queries and first
// keys arrive, and its first products run, while the unit before it ends.
//   warps 0-3, 4-7   softmax of tile 0, 1 (a thread owns a row: a lane of
//                    tensor memory), the rare rescaling of O, the results
//   warps 8-11       keys and values: the tiles K0 V0 K1 V1 .. into a ring of
//                    five slots: tile copies (TMA) of the pages' rows;
//                    16 bytes at a time where a tile ends beyond the sequence
//                    (those rows as zeros, so that what the cache holds there
//                    meets P = 0 as 0). e4m3 codes are copied to two tiles
//                    beside a ring of four slots and widened from there (keys
//                    to the queries' type, values to fp16)
//   warps 12, 13     the units (warp 12) and their queries: tile copies where
//                    the group divides 128, else 16 bytes at a time
//   warps 14, 15     tcgen05.mma of tile 0, 1: S from shared memory, O += P V
//                    with P read from tensor memory, where it takes the place
//                    of S
// Measured, back to back: 8192 rows of 64 heads over 8, fp16: 709 to 720 us
// (1530 to 1550 TFLOP/s, at the power limit; 624 with idle gaps); 140 to 700 rows
// behind 300 to 1500, 40 heads, bf16: 57 us; 37 rows of 32 heads: 8.2 us on the
// device, 9.2 a call. 8192 rows over e4m3 codes: fp16 queries 807 us, bf16 877.
// Head dim 64: 538 us
// (no pipe full: issue 49%, tensor 44%, exponentials 44%; a softmax warp's own
// 570 instructions per tile are the chain that binds).
// Where the units are fewer than the blocks, each is split over its keys into
// parts of at least kLeast tiles; the parts' (m, l, O) go to the workspace as
// fp32, and a second kernel joins them in their order. (Joined by the last
// part to arrive, 19 parts of 128 rows took one block longer than the parts
// themselves: 16 rows behind 30000 keys 55-76 us against 50.)
// Tensor memory: S0, S1 (128 columns each), O0, O1 (D each). Registers: 128 a
// thread at launch, 192 for the softmax warps and 64 for the rest (256 x 192
// + 256 x 64 = 512 x 128).
#include <type_traits>

#include "common.cuh"
#include "kernels.h"
#include "layer.cuh"
#include "tc_ptx.cuh"

namespace w4a16 {
namespace {

using namespace tc;

constexpr int kThreads = 512;
constexpr int kTile = 128;  // rows of a tile, and keys of a tile
constexpr int kMostSlots = 5;
constexpr int kPanel = kTile * 128;  // bytes of 64 dimensions of 128 rows
constexpr float kLog2e = 1.4426950408889634f, kLn2 = 0.6931471805599453f;
constexpr int kLeast = 4;    // key tiles of a part: as long as what a part costs beside them
constexpr float kSlack = 8.f;  // log2 of how far a row's maximum may run ahead

// barriers, [2]: of the row tiles, or of the two places of a unit's description
enum {
  kFull = 0,                   // [kSlots] a key or value tile is there
  kEmpty = kFull + kMostSlots, // [kSlots] both row tiles' products have read it
  kUnit = kEmpty + kMostSlots,     // [2] a unit is described
  kUnitFree = kUnit + 2,       // [2] every role has read it
  kQueries = kUnitFree + 2,    // [2] the queries are there
  kQueriesFree = kQueries + 2, // [2] the unit's last scores have read them
  kScores = kQueriesFree + 2,  // [2] S is there (and the last P V done)
  kProbs = kScores + 2,        // [2 parts][2] P is there
  kOut = kProbs + 4,           // [2] the unit's O is there
  kOutFree = kOut + 2,         // [2] O has been read
  kTurn = kOutFree + 2,        // [2] the tile's products may be issued
  kCopiers = kTurn + 2,        // the four copying warps meet
  kCodes = kCopiers + 1,       // [2] a tile of e4m3 codes is there
  kCodesFree = kCodes + 2,     // [2] it has been read
  kDrain = kCodesFree + 2,       // [2] products in flight, when giving up
  kBars = kDrain + 2
};
constexpr int kReaders = 8 + 4 + 1 + 2;  // warps that read a unit's description

struct Unit {
  int b, first, fresh, len;  // sequence, its first row, rows, cached tokens
  int row0, head;            // first of the unit's rows (tokens x heads), key/value head
  int j0, n[2];              // first key tile, and key tiles that the two row tiles need from it on
  int parts, part, slot;     // parts of the rows' keys, which one this is, and its place
  int valid;                 // 0: no unit is left
};

struct Control {
  uint64_t bars[kBars];
  Unit unit[2];
  uint32_t tmem;
  int abort;
};

template <int D>
constexpr int kTileBytes = D / 64 * kPanel;
template <int D>
constexpr int kSmem = (2 + kMostSlots) * kTileBytes<D> + (int)sizeof(Control) + 1024;
static_assert(kSmem<128> <= 227 * 1024, "one block's shared memory");

// A warp's part: O as [D / 4][32 rows] of four, maxima, sums, and the rows'
// places in the output (or -1).
template <int D>
constexpr int kPartFloats = 32 * (D + 3);
// The workspace's flag area, zero between calls: the queue, then from this
// byte on a count per place and warp of the parts to join from there on (0:
// none; a call that gave up before it had written a part joins nothing of
// it). 152 SMs' take 4.75 KiB.
constexpr size_t kFlagBytes = 32768, kJoinsAt = 256;

struct PromptArgs {
  AttnArgs a;
  int group;
  float mult;      // |scale| log2 e
  uint32_t negate;  // scale < 0
  int q_tiled;      // the map of the queries is there
  int* queue;       // next unit; at [2], 64 bits: blocks that are through << 32 | what they drew
  float* partial;   // [blocks][8 warps] of kPartFloats, where units can be split
  int* joins;       // [blocks][8 warps]
  size_t partial_floats;  // of the workspace's
  int most_parts;
};

__device__ __forceinline__ void tmem_ld32(uint32_t taddr, uint32_t (&r)[32]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x32.b32 "
      "{%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, "
      "%16, %17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31}, [%32];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]),
        "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15]), "=r"(r[16]),
        "=r"(r[17]), "=r"(r[18]), "=r"(r[19]), "=r"(r[20]), "=r"(r[21]), "=r"(r[22]), "=r"(r[23]), "=r"(r[24]),
        "=r"(r[25]), "=r"(r[26]), "=r"(r[27]), "=r"(r[28]), "=r"(r[29]), "=r"(r[30]), "=r"(r[31])
      : "r"(taddr));
}
__device__ __forceinline__ void tmem_st16(uint32_t taddr, const uint32_t (&r)[16]) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], "
      "{%1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, %16};" ::"r"(taddr),
      "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]), "r"(r[9]),
      "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15])
      : "memory");
}
__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
// Two fp32 lanes of one 64-bit register.
__device__ __forceinline__ uint64_t pack2(float lo, float hi) {
  uint64_t v;
  asm("mov.b64 %0, {%1, %2};" : "=l"(v) : "f"(lo), "f"(hi));
  return v;
}
__device__ __forceinline__ void unpack2(uint64_t v, float& lo, float& hi) {
  asm("mov.b64 {%0, %1}, %2;" : "=f"(lo), "=f"(hi) : "l"(v));
}
__device__ __forceinline__ uint64_t fma2(uint64_t a, uint64_t b, uint64_t c) {
  uint64_t d;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(d) : "l"(a), "l"(b), "l"(c));
  return d;
}
__device__ __forceinline__ uint64_t add2(uint64_t a, uint64_t b) {
  uint64_t d;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(a), "l"(b));
  return d;
}
// Keeps the uses of loaded tensor-memory registers behind the wait for them.
__device__ __forceinline__ void tie(uint32_t (&r)[32]) {
  asm volatile(""
               : "+r"(r[0]), "+r"(r[1]), "+r"(r[2]), "+r"(r[3]), "+r"(r[4]), "+r"(r[5]), "+r"(r[6]), "+r"(r[7]),
                 "+r"(r[8]), "+r"(r[9]), "+r"(r[10]), "+r"(r[11]), "+r"(r[12]), "+r"(r[13]), "+r"(r[14]), "+r"(r[15]),
                 "+r"(r[16]), "+r"(r[17]), "+r"(r[18]), "+r"(r[19]), "+r"(r[20]), "+r"(r[21]), "+r"(r[22]), "+r"(r[23]),
                 "+r"(r[24]), "+r"(r[25]), "+r"(r[26]), "+r"(r[27]), "+r"(r[28]), "+r"(r[29]), "+r"(r[30]), "+r"(r[31]));
}
__device__ __forceinline__ void tie(uint32_t (&r)[16]) {
  asm volatile(""
               : "+r"(r[0]), "+r"(r[1]), "+r"(r[2]), "+r"(r[3]), "+r"(r[4]), "+r"(r[5]), "+r"(r[6]), "+r"(r[7]),
                 "+r"(r[8]), "+r"(r[9]), "+r"(r[10]), "+r"(r[11]), "+r"(r[12]), "+r"(r[13]), "+r"(r[14]), "+r"(r[15]));
}
__device__ __forceinline__ void cp16(uint32_t dst, const void* src, bool valid) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(valid ? 16 : 0) : "memory");
}
__device__ __forceinline__ void cp_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void cp_wait() { asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory"); }

// Byte offset of 16-byte chunk c of row r in a tile: panels of 64 dimensions
// with the 128-byte swizzle.
__device__ __forceinline__ uint32_t chunk_at(int r, int c) {
  return (uint32_t)((c >> 3) * kPanel + r * 128 + (((c & 7) ^ (r & 7)) << 4));
}

// The row of a key, or 0 for one beyond the sequence (whose page is not looked up).
template <class F>
__device__ __forceinline__ unsigned long long row_of_or_0(const F& row_of, int key, int len) {
  return key < len ? row_of(key) : 0ull;
}

// Bounded wait for the phase of parity `parity`, as mbar_wait's, by waits
// that the hardware suspends for up to kNap: most of this kernel's warps wait
// most of the time, and polling would take the issue slots of the softmax
// warps beside them.
constexpr uint32_t kNap = 20000;  // ns
__device__ __forceinline__ bool nap_wait(uint32_t bar, uint32_t parity, volatile int* abort_flag, int code, int* err) {
  auto nap = [&]() {
    uint32_t ok;
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "mbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2, %3;\n\t"
        "selp.u32 %0, 1, 0, p;\n\t}"
        : "=r"(ok)
        : "r"(bar), "r"(parity), "r"(kNap)
        : "memory");
    return ok != 0;
  };
  if (nap()) return true;
  const uint64_t t0 = globaltimer();
  while (true) {
    if (nap()) return true;
    if (*abort_flag) return false;
    if (globaltimer() - t0 > kWaitLimitNs) {
      *abort_flag = 1;
      atomicOr(err, code);
      return false;
    }
  }
}

// True in one lane of the (converged) warp.
__device__ __forceinline__ bool elect_one() {
  uint32_t ok;
  asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.u32 %0, 1, 0, p;\n\t}" : "=r"(ok));
  return ok != 0;
}

// tcgen05.mma kind::f16 with A and B (ss), or B alone (ts: A in tensor
// memory), given by the lower halves of their shared-memory descriptors. Both
// kinds of tiles have the same upper half: 8-row groups 1024 bytes apart
// (stride byte offset), 128-byte swizzle. The queries and keys are K-major;
// the values are read with the dimensions innermost (MN-major: 8-key groups at
// the stride byte offset, panels of 64 dimensions at the leading one).
__device__ __forceinline__ void mma_ss(uint32_t d, uint32_t a_lo, uint32_t b_lo, uint32_t hi, uint32_t idesc, bool add) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t.reg .b64 da, db;\n\t"
      "mov.b64 da, {%1, %3};\n\tmov.b64 db, {%2, %3};\n\t"
      "setp.ne.b32 p, %5, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], da, db, %4, p;\n\t}" ::"r"(d),
      "r"(a_lo), "r"(b_lo), "r"(hi), "r"(idesc), "r"((uint32_t)add)
      : "memory");
}
__device__ __forceinline__ void mma_ts(uint32_t d, uint32_t a, uint32_t b_lo, uint32_t hi, uint32_t idesc, bool add) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t.reg .b64 db;\n\t"
      "mov.b64 db, {%2, %3};\n\t"
      "setp.ne.b32 p, %5, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], db, %4, p;\n\t}" ::"r"(d),
      "r"(a), "r"(b_lo), "r"(hi), "r"(idesc), "r"((uint32_t)add)
      : "memory");
}

__device__ __forceinline__ uint2 lds64(uint32_t addr) {
  uint2 v;
  asm volatile("ld.shared.v2.u32 {%0, %1}, [%2];" : "=r"(v.x), "=r"(v.y) : "r"(addr));
  return v;
}

// Eight e4m3 codes to fp16 (exact).
__device__ __forceinline__ uint4 widen(uint32_t lo, uint32_t hi) {
  uint4 v;
  e4m3x4_to_half2x2(lo, v.x, v.y);
  e4m3x4_to_half2x2(hi, v.z, v.w);
  return v;
}

// And to bf16 (exact).
__device__ __forceinline__ uint4 widen_bf16(uint32_t lo, uint32_t hi) {
  const uint4 h = widen(lo, hi);
  const float2 a = unpack16<false>(h.x), b = unpack16<false>(h.y), c = unpack16<false>(h.z), d = unpack16<false>(h.w);
  return make_uint4(pack16<true>(a.x, a.y), pack16<true>(b.x, b.y), pack16<true>(c.x, c.y), pack16<true>(d.x, d.y));
}

// kB: 16-bit values are bf16, else fp16; k8: e4m3 cache. The scores' product
// is in the queries' type, P V in the cache's or, over e4m3 codes, in fp16
// (both types hold every code).
template <bool kB, bool k8, int D>
__global__ void __launch_bounds__(kThreads, 1) attn_prompt_kernel(const PromptArgs p, const __grid_constant__ CUtensorMap map_k,
                                                                 const __grid_constant__ CUtensorMap map_v,
                                                                 const __grid_constant__ CUtensorMap map_q) {
  constexpr int kBytes = kTileBytes<D>;
  constexpr bool kP = kB && !k8;  // P V in bf16
  constexpr int kChunks = D / 8;  // 16-byte chunks of a row
  constexpr int kSlots = k8 ? kMostSlots - 1 : kMostSlots;  // (two tiles of codes in place of one)
  extern __shared__ uint8_t smem_raw[];
  const uint32_t raw = (uint32_t)__cvta_generic_to_shared(smem_raw);
  const uint32_t base = (raw + 1023u) & ~1023u;  // queries [2], ring [kSlots]
  const uint32_t ring = base + 2 * kBytes, codes = ring + kSlots * kBytes;
  Control& ctl = *reinterpret_cast<Control*>(smem_raw + (ring - raw) + kMostSlots * kBytes);
  const uint32_t bars = (uint32_t)__cvta_generic_to_shared(&ctl.bars[0]);
  auto bar = [&](int i) { return bars + 8u * (uint32_t)i; };
  const AttnArgs& a = p.a;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  volatile int* abort_flag = &ctl.abort;

  if (tid == 0) {
    for (int i = 0; i < kSlots; ++i) {
      mbar_init(bar(kFull + i), k8 ? 128 : 1);
      mbar_init(bar(kEmpty + i), 2);
    }
    for (int t = 0; t < 2; ++t) {
      mbar_init(bar(kUnit + t), 1);
      mbar_init(bar(kUnitFree + t), kReaders);
      mbar_init(bar(kQueries + t), p.q_tiled ? 1 : 64);
      mbar_init(bar(kQueriesFree + t), 1);
      mbar_init(bar(kScores + t), 1);
      mbar_init(bar(kProbs + t), 128);
      mbar_init(bar(kProbs + 2 + t), 128);
      mbar_init(bar(kOut + t), 1);
      mbar_init(bar(kOutFree + t), 128);
      mbar_init(bar(kTurn + t), 1);
      mbar_init(bar(kCodes + t), 1);
      mbar_init(bar(kCodesFree + t), 128);
      mbar_init(bar(kDrain + t), 1);
    }
    mbar_init(bar(kCopiers), 128);
    ctl.abort = 0;
    fence_barrier_init();
  }
  if (warp == 12) {
    tmem_alloc((uint32_t)__cvta_generic_to_shared(&ctl.tmem), 512);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = ctl.tmem;
  allow_dependent_launch();
  grid_dependency_wait();

  // The u-th unit of this block.
  Unit unit;
  int most = 0;
  auto read_unit = [&](int u) {
    unit = ctl.unit[u & 1];
    most = max(unit.n[0], unit.n[1]);
    return unit.valid != 0;
  };
  // A wait of a whole warp: all of its lanes go on, or none.
  auto warp_wait = [&](int i, uint32_t phase, int code) {
    return __all_sync(0xffffffffu, nap_wait(bar(i), phase, abort_flag, code, a.err)) != 0;
  };
  auto next_unit = [&](int u, int code, bool release) {  // of a whole warp
    if (!warp_wait(kUnit + (u & 1), (uint32_t)(u >> 1) & 1u, code)) return false;
    const bool valid = read_unit(u);
    __syncwarp();
    if (valid && release && lane == 0) mbar_arrive(bar(kUnitFree + (u & 1)));
    return valid;
  };

  if (warp < 8) {
    asm volatile("setmaxnreg.inc.sync.aligned.u32 192;");
    const int t = warp >> 2;
    const uint32_t lanes = (uint32_t)(warp & 3) << 21;  // the warp's quarter of the lanes
    const uint32_t scores = tmem + lanes + (uint32_t)(t * kTile), out = tmem + lanes + 256u + (uint32_t)(t * D);
    uint32_t score_phase = 0, out_phase = 0;
    bool ok = true;
    for (int u = 0; ok; ++u) {
      // (read where it is needed, and released at the end: registers are short)
      if (!warp_wait(kUnit + (u & 1), (uint32_t)(u >> 1) & 1u, kErrEpilogue)) break;
      const Unit& unit = ctl.unit[u & 1];
      if (!unit.valid) break;
      const int nt = unit.n[t];
      const int row = unit.row0 + t * kTile + (tid & 127);
      const bool live = row < unit.fresh * p.group;
      const int token = live ? row / p.group : 0, head = unit.head * p.group + (live ? row - token * p.group : 0);
      // keys of the unit's that this row sees (rows beyond the sequence mask
      // nothing: what they give is not written)
      const int limit = live ? unit.len - unit.fresh + token + 1 - unit.j0 * kTile : 0x7fffffff;
      const bool idle = __all_sync(0xffffffffu, !live);
      int to = live ? (unit.first + token) * a.heads + head : -1;
      const float mult = k8 ? positive(p.mult * *ld_at(a.cache.k_scale + unit.head, a.cache.k_scale, (size_t)a.cache.kv_heads, a.err)) : p.mult;
      float m = -INFINITY, l = 0.f;
      for (int j = 0; j < nt; ++j) {
        if (!(ok = warp_wait(kScores + t, score_phase, kErrEpilogue))) break;
        score_phase ^= 1u;
        if (idle) {  // no row of this warp's: P is left as it is
          mbar_arrive(bar(kProbs + t));
          mbar_arrive(bar(kProbs + 2 + t));
          continue;
        }
        tc_fence_after();
        uint32_t s[4][32];
        in_tmem((uint32_t)(t * kTile), kTile, 512, a.err);
#pragma unroll
        for (int q = 0; q < 4; ++q) tmem_ld32(scores + 32 * q, s[q]);
        tmem_wait_ld();
#pragma unroll
        for (int q = 0; q < 4; ++q) tie(s[q]);
        // masked 32 keys at a time, where a row of the warp needs it
        const int seen = limit - j * kTile;
        if (!__all_sync(0xffffffffu, seen >= kTile)) {
#pragma unroll
          for (int q = 0; q < 4; ++q) {
            const int left = seen - 32 * q;
            if (__all_sync(0xffffffffu, left >= 32)) continue;
#pragma unroll
            for (int i = 0; i < 32; ++i)
              if (i >= left) s[q][i] = 0xff800000u;
          }
        }
        float top4[4];
#pragma unroll
        for (int q = 0; q < 4; ++q) top4[q] = fmaxf(__uint_as_float(s[q][0]), __uint_as_float(s[q][1]));
#pragma unroll
        for (int i = 2; i < 32; i += 2)
#pragma unroll
          for (int q = 0; q < 4; ++q)
            top4[q] = fmaxf(fmaxf(top4[q], __uint_as_float(s[q][i])), __uint_as_float(s[q][i + 1]));
        const float top = fmaxf(fmaxf(top4[0], top4[1]), fmaxf(top4[2], top4[3])) * mult;
        const bool moves = top > m + kSlack;
        if (__any_sync(0xffffffffu, moves)) {
          const float f = moves ? ex2(m - top) : 1.f;
          if (moves) m = top;
          l *= f;
          if (j > 0) {
            // the scores' arrival says that the product with the last P is done
#pragma unroll 1
            for (int c = 0; c < D; c += 16) {
              uint32_t o[16];
              tmem_ld16(out + c, o);
              tmem_wait_ld();
              tie(o);
#pragma unroll
              for (int i = 0; i < 16; ++i) o[i] = __float_as_uint(__uint_as_float(o[i]) * f);
              tmem_st16(out + c, o);
            }
          }
        }
        const float shift = m == -INFINITY ? 0.f : -m;
        // P in two parts, of 96 and 32 keys: the product with the first runs
        // while the second is formed; the sums wait until both are on their
        // way. P is rounded to 16 bits (relative 2^-11, or 2^-8 with bf16
        // values; fp16 has fewer bits for terms below 2^-14 of m and none below
        // 2^-25, which the sums take whole: with one key 2^26 above 8192 others
        // the result is 2^-13 low).
        const uint64_t mult2 = pack2(mult, mult), shift2 = pack2(shift, shift);
#pragma unroll
        for (int part = 0; part < 2; ++part) {
#pragma unroll
          for (int q = part ? 3 : 0; q < (part ? 4 : 3); ++q) {
            uint32_t w[16];
#pragma unroll
            for (int i = 0; i < 16; ++i) {
              float x, y;
              unpack2(fma2(pack2(__uint_as_float(s[q][2 * i]), __uint_as_float(s[q][2 * i + 1])), mult2, shift2), x, y);
              x = ex2(x), y = ex2(y);
              s[q][2 * i] = __float_as_uint(x), s[q][2 * i + 1] = __float_as_uint(y);
              w[i] = pack16<kP>(x, y);
            }
            tmem_st16(scores + 16 * q, w);
          }
          tmem_wait_st();
          tc_fence_before();
          mbar_arrive(bar(kProbs + 2 * part + t));
        }
        uint64_t l4[4] = {0, 0, 0, 0};
#pragma unroll
        for (int i = 0; i < 32; i += 2)
#pragma unroll
          for (int q = 0; q < 4; ++q) l4[q] = add2(l4[q], pack2(__uint_as_float(s[q][i]), __uint_as_float(s[q][i + 1])));
        float lo, hi;
        unpack2(add2(add2(l4[0], l4[1]), add2(l4[2], l4[3])), lo, hi);
        l += lo + hi;
      }
      if (ok && nt > 0) {
        ok = warp_wait(kOut + t, out_phase, kErrEpilogue);
        out_phase ^= 1u;
        tc_fence_after();
      }
      if (!ok) break;
      // (Loops: code that runs once per unit is fetched anew every time.)
      in_tmem(256u + (uint32_t)(t * D), D, 512, a.err);
      float* mine = p.partial + (size_t)(unit.slot * 8 + warp) * kPartFloats<D>;
      if (unit.parts > 1) {
        if (!idle && in_buf(mine + kPartFloats<D> - 1, p.partial, p.partial_floats, a.err) &&
            in_buf(p.joins + unit.slot * 8 + warp, p.joins, (kFlagBytes - kJoinsAt) / sizeof(int), a.err)) {
          if (nt > 0) {
#pragma unroll 1
            for (int d0 = 0; d0 < D; d0 += 32) {
              uint32_t o[32];
              tmem_ld32(out + d0, o);
              tmem_wait_ld();
              tie(o);
#pragma unroll
              for (int i = 0; i < 8; ++i)
                reinterpret_cast<uint4*>(mine)[(d0 / 4 + i) * 32 + lane] = make_uint4(o[4 * i], o[4 * i + 1], o[4 * i + 2], o[4 * i + 3]);
            }
          }
          mine[32 * D + lane] = m;
          mine[32 * (D + 1) + lane] = l;
          reinterpret_cast<int*>(mine)[32 * (D + 2) + lane] = to;
          if (unit.part == 0 && lane == 0) p.joins[unit.slot * 8 + warp] = unit.parts;
        }
        to = -1;  // written by the joining kernel
      } else {
        // (a sum of zero: no key has weight; a NaN sum is the row's result)
        const float inv = l == 0.f ? 0.f : (k8 ? *ld_at(a.cache.v_scale + unit.head, a.cache.v_scale, (size_t)a.cache.kv_heads, a.err) : 1.f) / l;
#pragma unroll 2
        for (int d0 = 0; d0 < D; d0 += 32) {
          uint32_t o[32];
          if (nt > 0) {
            tmem_ld32(out + d0, o);
            tmem_wait_ld();
            tie(o);
          }
          // transposed among four lanes (a lane's four 16-byte chunks of its
          // row become one chunk of four rows), so that whole sectors are
          // written: a row per lane would be 32 lines per store
          uint32_t x[4][4];
#pragma unroll
          for (int i = 0; i < 16; ++i)
            x[i / 4][i & 3] = l == 0.f ? 0 : pack16<kB>(__uint_as_float(o[2 * i]) * inv, __uint_as_float(o[2 * i + 1]) * inv);
#pragma unroll
          for (int bit = 1; bit < 4; bit <<= 1)
#pragma unroll
            for (int i = 0; i < 4; ++i)
              if (!(i & bit)) {
                const bool upper = lane & bit;
#pragma unroll
                for (int k = 0; k < 4; ++k) {
                  const uint32_t got = __shfl_xor_sync(0xffffffffu, upper ? x[i][k] : x[i | bit][k], bit);
                  x[i][k] = upper ? got : x[i][k];
                  x[i | bit][k] = upper ? x[i | bit][k] : got;
                }
              }
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const int place = __shfl_sync(0xffffffffu, to, (lane & 28) + i);
            if (place >= 0 && in_buf(a.out + (size_t)place * D + d0 + (lane & 3) * 8, a.out, (size_t)a.rows * a.heads * D - 7, a.err))
              *reinterpret_cast<uint4*>(a.out + (size_t)place * D + d0 + (lane & 3) * 8) = make_uint4(x[i][0], x[i][1], x[i][2], x[i][3]);
          }
        }
      }
      if (nt > 0) {  // O is read: the next unit may write it
        tc_fence_before();
        mbar_arrive(bar(kOutFree + t));
      }
      if (to >= 0 && a.lse && in_buf(a.lse + to, a.lse, (size_t)a.rows * a.heads, a.err)) a.lse[to] = l == 0.f ? -INFINITY : m * kLn2 + logf(l);
      __syncwarp();
      if (lane == 0) mbar_arrive(bar(kUnitFree + (u & 1)));
    }
  } else {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 64;");
    if (warp < 12) {
      const int v = tid - 256;
      const int shift = a.cache.page_shift, mask = (1 << shift) - 1;
      bool ok = true;
      int count = 0;   // tiles so far
      int copied = 0;  // those before which this warp's tile copies have been issued
      uint32_t met = 0;
      auto slot_of = [&]() { return count % kSlots; };
      auto wait_slot = [&]() {
        return count < kSlots || warp_wait(kEmpty + count % kSlots, (uint32_t)(count / kSlots - 1) & 1u, kErrProducer);
      };
      auto meet = [&]() {  // of the four copying warps, bounded
        mbar_arrive(bar(kCopiers));
        ok = warp_wait(kCopiers, met, kErrProducer) && ok;
        met ^= 1u;
      };
      for (int u = 0; ok; ++u) {
        if (!next_unit(u, kErrProducer, true)) break;
        const int len = unit.len;
        // the first row, in the cache seen as rows of D values, of this head's
        // place of key `key` of the sequence
        auto row_of = [&](int key) {
          return (((unsigned long long)page_of(a, unit.b, key >> shift) * a.cache.kv_heads + unit.head) << shift) + (key & mask);
        };
        // a tile copy's first row and its place: as they are, or (checked
        // build) 0 and the first slot, recorded, where it would leave them
        auto first_row = [&](unsigned long long row, int n) {
          if (!kCheckedBuild || row + n <= cache_rows(a.cache)) return (int)row;
          atomicOr(a.err, kErrBounds);
          return 0;
        };
        auto slot_at = [&](uint32_t at, uint32_t bytes) { return in_smem(at, bytes, raw, a.err) ? at : ring; };
        if (!k8) {
          // tiles that lie inside the sequence: tile copies of the pages' rows,
          // a lane for each page and panel. Small pages' copies (16 of them
          // for 16 tokens) are shared among the four warps: a warp issues its
          // lanes' copies one after another.
          const int whole = max(0, min(most, len / kTile - unit.j0));
          const int end = count + 2 * whole;
          const int box = min(1 << shift, kTile), boxes = kTile / box, copies = D / 64 * boxes;
          const int sharing = copies > 4 ? 4 : 1, each = copies / sharing;
          if (warp - 8 < sharing) {
            const int mine = (warp - 8) * each + lane, panel = mine / boxes, part = mine % boxes;
            // the page of the next tile is looked up while this one is waited for
            unsigned long long row = 0, ahead = whole > 0 ? row_of(unit.j0 * kTile + part * box) : 0;
            for (int j = 0; count < end && ok; ++count) {
              const bool values = (end - count) & 1;
              if (!values) {
                row = ahead;
                if (++j < whole) ahead = row_of((unit.j0 + j) * kTile + part * box);
              }
              if (!(ok = wait_slot())) break;
              const uint32_t full = bar(kFull + slot_of());
              if (mine == 0) mbar_expect_tx(full, kBytes);
              __syncwarp();
              if (lane < each)
                tma_load_2d(slot_at(ring + slot_of() * kBytes, kBytes) + panel * kPanel + part * box * 128, values ? &map_v : &map_k,
                            panel * 64, first_row(row, box), full);
              copied = count + 1;
            }
          }
          if (ok) count = end;
          // the ragged last tile: 16 bytes at a time, rows beyond the sequence
          // as zeros
          if (whole < most) {
            meet();  // the first warp has come as far: a slot's phase is known
            const int r0 = v / kChunks, c = v % kChunks;
            constexpr int kStride = 128 / kChunks;
            for (int j = whole; j < most && ok; ++j) {
              const int key0 = (unit.j0 + j) * kTile;
              const unsigned long long group = row_of_or_0(row_of, key0 + 16 * (lane & 7), len);
              int slots[2];
#pragma unroll 1
              for (int kv = 0; kv < 2 && ok; ++kv) {
                if (!(ok = wait_slot())) break;
                const uint8_t* src = static_cast<const uint8_t*>(kv ? a.cache.v : a.cache.k);
                const uint32_t dst = ring + slot_of() * kBytes + chunk_at(r0, c);
#pragma unroll 4
                for (int x = 0; x < kTile / kStride; ++x) {
                  const int r = r0 + x * kStride;
                  const unsigned long long row = __shfl_sync(0xffffffffu, group, r >> 4) + (r & 15);
                  const bool valid = key0 + r < len;
                  const uint8_t* from = valid ? ld_at(src + row * (2 * D) + c * 16, src, cache_rows(a.cache) * (2 * D) - 15, a.err) : src;
                  if (in_smem(dst + x * kStride * 128, 16, raw, a.err)) cp16(dst + x * kStride * 128, from, valid);
                }
                cp_commit();
                slots[kv] = slot_of();
                ++count;
              }
              // the keys, then the values
              cp_wait<1>();
              fence_async_shared();
              meet();
              if (v == 0 && ok) mbar_arrive(bar(kFull + slots[0]));
              cp_wait<0>();
              fence_async_shared();
              meet();
              if (v == 0 && ok) mbar_arrive(bar(kFull + slots[1]));
            }
          }
        } else {
          // tile copies of the pages' codes, up to two tiles ahead; then a thread
          // widens the 8-code chunk c of the rows r0 + x * kStride (eight lanes
          // then write the eight chunks of one row of a panel: no bank twice)
          constexpr int kPieces = D / 8, kStride = 128 / kPieces, kLoads = kTile / kStride;
          const int r0 = v / kPieces, c = v % kPieces;
          const int box = min(1 << shift, kTile), boxes = kTile / box;
          const int sharing = boxes >= 4 ? 4 : 1, each = boxes / sharing, mine = (warp - 8) * each + lane;
          // (the page of the next tile is looked up while this one is copied)
          auto look = [&](int j) { return row_of_or_0(row_of, (unit.j0 + j) * kTile + min(mine, boxes - 1) * box, len); };
          unsigned long long row = 0, ahead = most > 0 ? look(0) : 0;
          const int start = count;
          auto copy = [&](int i) {  // tile i of the unit
            const int n = start + i, at = n & 1;
            if (!(i & 1)) {
              row = ahead;
              if (i / 2 + 1 < most) ahead = look(i / 2 + 1);
            }
            if (n >= 2 && !warp_wait(kCodesFree + at, (uint32_t)(n / 2 - 1) & 1u, kErrProducer)) return false;
            if (mine == 0) mbar_expect_tx(bar(kCodes + at), kTile * D);
            __syncwarp();
            if (lane < each)
              tma_load_2d(slot_at(codes + at * (kTile * D), kTile * D) + mine * box * D, i & 1 ? &map_v : &map_k, 0,
                          first_row(row, box), bar(kCodes + at));
            copied = n + 1;
            return true;
          };
          if (most > 0 && warp - 8 < sharing) ok = copy(0) && copy(1);
          for (int i = 0; i < 2 * most && ok; ++i, ++count) {
            const int key0 = (unit.j0 + (i >> 1)) * kTile, at = count & 1;
            const bool inside = key0 + kTile <= len;
            if (!(ok = warp_wait(kCodes + at, (uint32_t)(count / 2) & 1u, kErrProducer))) break;
            // kGroup rows are loaded while those before them are widened and
            // stored: the pass is a chain of waits on the shared memory that
            // the MMAs keep busy, not a matter of issue (all rows first: 890 us
            // against 778 at 1 x 8192; bf16 keys have registers for two rows)
            constexpr int kGroup = kB ? 2 : 4;
            uint2 x2[2][kGroup];
            auto load = [&](int g) {
#pragma unroll
              for (int x = 0; x < kGroup; ++x) {
                const int r = r0 + (g * kGroup + x) * kStride;
                x2[g & 1][x] = lds64(codes + at * (kTile * D) + r * D + c * 8);
                if (!inside && key0 + r >= len) x2[g & 1][x] = make_uint2(0, 0);
              }
            };
            load(0);
            if (!(ok = wait_slot())) break;
            const uint32_t to = slot_at(ring + slot_of() * kBytes, kBytes) + chunk_at(r0, c);
            auto groups = [&](auto b16) {
#pragma unroll
              for (int g = 0; g < kLoads / kGroup; ++g) {
                if (g + 1 < kLoads / kGroup) {
                  load(g + 1);
                } else {
                  mbar_arrive(bar(kCodesFree + at));
                  if (i + 2 < 2 * most && warp - 8 < sharing) ok = copy(i + 2);
                }
#pragma unroll
                for (int x = 0; x < kGroup; ++x) {  // kStride is a multiple of 8: the swizzle stays
                  const uint2 y = x2[g & 1][x];
                  const uint4 w = decltype(b16)::value ? widen_bf16(y.x, y.y) : widen(y.x, y.y);
                  sts128(to + (g * kGroup + x) * kStride * 128, w.x, w.y, w.z, w.w);
                }
              }
            };
            if (kB && !(i & 1)) groups(std::true_type{}); else groups(std::false_type{});
            fence_async_shared();
            mbar_arrive(bar(kFull + slot_of()));
          }
        }
      }
      cp_wait<0>();
      // no copy may land after this CTA has left, whatever ended its work (a
      // slot that has been filled again since was read before: it had landed)
      for (int n = k8 ? count : max(0, count - kSlots); n < copied; ++n) {
        if (k8)
          mbar_drain(bar(kCodes + (n & 1)), (uint32_t)(n / 2) & 1u, a.err);
        else
          mbar_drain(bar(kFull + n % kSlots), (uint32_t)(n / kSlots) & 1u, a.err);
      }
    } else if (warp < 14) {
      // Warp 12 takes units from the queue, numbered from the last rows of the
      // last sequence on, a key/value head after another. It walks back over
      // the sequences, 32 at a time: v units of this lane's sequence, `upto`
      // of the group's up to it, `before` of the groups before.
      int first = 0, fresh = 0, len = 0, v = 0, upto = 0, group = 0, before = 0, total = 0;
      auto look = [&]() {
        const int b = 32 * group + lane;
        first = fresh = len = v = 0;
        if (b < a.batch) {
          const int s0 = *ld_at(a.starts + b, a.starts, (size_t)a.batch + 1, a.err);
          const int s1 = *ld_at(a.starts + b + 1, a.starts, (size_t)a.batch + 1, a.err);
          const int n0 = *ld_at(a.lens + b, a.lens, (size_t)a.batch, a.err);
          first = checked(a, s0, a.rows);
          fresh = checked(a, s1, a.rows) - first;
          if (fresh < 0) {
            atomicOr(a.err, kErrRange);
            fresh = 0;
          }
          len = checked(a, n0, (int)min((long long)a.max_pages << a.cache.page_shift, 0x7fffffffll));
          v = (int)(((long long)fresh * p.group + 2 * kTile - 1) / (2 * kTile));
        }
        upto = v;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
          const int x = __shfl_up_sync(0xffffffffu, upto, o);
          if (lane >= o) upto += x;
        }
      };
      const int groups = (a.batch + 31) / 32;
      if (warp == 12) {
        for (group = 0; group < groups; ++group) {
          before = total;
          look();
          total += __shfl_sync(0xffffffffu, upto, 31);
        }
        --group;
      }
      // parts per unit: as many as there are blocks for. (Two rounds of more and
      // smaller parts, where that is shorter, gained 2% at 300 rows behind 4000
      // of 64 heads over 8: 80 units on 152 blocks.)
      const int count = total * a.cache.kv_heads, grid = (int)gridDim.x;
      const int split = count > 0 && count < grid ? max(1, min(grid / count, p.most_parts)) : 1;
      const int w = tid - 384, c = w % kChunks;
      constexpr int kStride = 64 / kChunks;
      const int step_head = kStride % p.group;
      const long long step = (long long)(kStride / p.group) * a.ldq + step_head * D, wrap = a.ldq - (long long)p.group * D;
      bool ok = true;
      int asked = 0;  // tile copies of queries, alternately of tile 0 and 1
      uint32_t drawn = 0;  // numbers that this block took from the queue
      for (int u = 0; ok; ++u) {
        if (warp == 12) {
          if (u >= 2 && !(ok = warp_wait(kUnitFree + (u & 1), (uint32_t)(u / 2 - 1) & 1u, kErrProducer))) break;
          Unit& to = ctl.unit[u & 1];
          for (bool found = false; !found;) {
            int i = 0;
            if (lane == 0) i = atomicAdd(p.queue, 1);
            i = __shfl_sync(0xffffffffu, i, 0);
            ++drawn;
            // (a queue that was negative ends the block's work, it does not search)
            if (i < 0 && lane == 0) atomicOr(a.err, kErrWorkspace);
            const int id = i / split, want = i < 0 ? -1 : total - 1 - id / a.cache.kv_heads;
            if (want < 0) {
              if (lane == 0) to.valid = 0;
              break;
            }
            while (want < before) {
              --group;
              look();
              before -= __shfl_sync(0xffffffffu, upto, 31);
            }
            const int lo = before + upto - v;
            bool mine = false;
            if (lo <= want && want < lo + v) {
              const int row0 = (want - lo) * (2 * kTile), rows = fresh * p.group;  // rows: at most 2^30
              int n[2];
#pragma unroll
              for (int t = 0; t < 2; ++t) {  // up to the last row's position
                const int from = row0 + t * kTile, past = min(from + kTile, rows);
                const int last = from < past ? len - fresh + (past - 1) / p.group : -1;
                n[t] = last < 0 ? 0 : last / kTile + 1;
              }
              const int all = max(n[0], n[1]), parts = max(1, min(split, all / kLeast)), part = i % split;
              if (part < parts) {  // (a short unit has fewer parts than there are places)
                // (products below 2^31: at most 2^23 tiles, parts up to the blocks)
                const int j0 = parts == 1 ? 0 : part * all / parts, j1 = parts == 1 ? all : (part + 1) * all / parts;
                to = {32 * group + lane, first, fresh, len, row0, id % a.cache.kv_heads, j0,
                      {max(0, min(n[0], j1) - j0), max(0, min(n[1], j1) - j0)}, parts, part, i, 1};
                mine = true;
              }
            }
            found = __any_sync(0xffffffffu, mine);
          }
          __syncwarp();
          if (lane == 0) mbar_arrive(bar(kUnit + (u & 1)));
        }
        if (!next_unit(u, kErrProducer, warp == 13)) break;
        if (p.q_tiled) {
          // whole tokens to a tile: a tile copy of [tokens][heads][D]; rows
          // beyond the sequence's are of no use and do no harm
          if (warp == 13) {
#pragma unroll 1
            for (int t = 0; t < 2 && ok; ++t) {
              if (u > 0 && !(ok = warp_wait(kQueriesFree + t, (uint32_t)(u - 1) & 1u, kErrProducer))) break;
              if (lane == 0) {
                mbar_expect_tx(bar(kQueries + t), kBytes);
#pragma unroll
                for (int d = 0; d < D / 64; ++d)
                  tma_load_3d((in_smem(base + t * kBytes, kBytes, raw, a.err) ? base + t * kBytes : base) + d * kPanel, &map_q, d * 64, unit.head * p.group,
                              unit.first + (unit.row0 + t * kTile) / p.group, bar(kQueries + t));
              }
              ++asked;
              __syncwarp();
            }
          }
          continue;
        }
        // else a thread copies chunk c of every kStride-th row
        int row = unit.row0 + w / kChunks, head = row % p.group;
        const uint16_t* src =
            a.q + (size_t)(unit.first + row / p.group) * a.ldq + (size_t)(unit.head * p.group + head) * D + c * 8;
#pragma unroll 1
        for (int t = 0; t < 2 && ok; ++t) {
          if (u > 0 && !(ok = warp_wait(kQueriesFree + t, (uint32_t)(u - 1) & 1u, kErrProducer))) break;
#pragma unroll 4
          for (int r = w / kChunks; r < kTile; r += kStride) {
            const bool valid = row < unit.fresh * p.group;
            const uint32_t dst = base + t * kBytes + chunk_at(r, c);
            const uint16_t* from = valid ? ld_at(src, a.q, span(a.rows, a.ldq, a.heads * D) - 7, a.err) : a.q;
            if (in_smem(dst, 16, raw, a.err)) cp16(dst, from, valid);
            row += kStride;
            src += step;
            head += step_head;
            if (head >= p.group) {
              head -= p.group;
              src += wrap;
            }
          }
          cp_commit();
          if (t == 1) {
            cp_wait<1>();
            fence_async_shared();
            mbar_arrive(bar(kQueries));
            cp_wait<0>();
            fence_async_shared();
            mbar_arrive(bar(kQueries + 1));
          }
        }
        __syncwarp();
      }
      // Every block comes here once, whatever ended its work; the last one
      // leaves the queue zero. The blocks draw every part's number and one
      // more each: another sum is that of a queue that was not zero before the
      // call (or of a block that gave up), whose call has left rows out.
      if (warp == 12 && lane == 0) {
        const unsigned long long all =
            atomicAdd(reinterpret_cast<unsigned long long*>(p.queue + 2), (1ull << 32) | drawn) + ((1ull << 32) | drawn);
        if ((int)(all >> 32) == grid) {
          if ((uint32_t)all != (uint32_t)max(count, 0) * split + grid) atomicOr(a.err, kErrWorkspace);
          p.queue[0] = p.queue[2] = p.queue[3] = 0;
        } else if ((uint32_t)(all >> 32) > (uint32_t)grid) {
          atomicOr(a.err, kErrWorkspace);
        }
      }
      cp_wait<0>();
      for (int n = max(0, asked - 2); n < asked; ++n) mbar_drain(bar(kQueries + (n & 1)), (uint32_t)(n / 2) & 1u, a.err);
    } else if (elect_one()) {
      // one warp per row tile, one thread of it
      constexpr uint32_t kDescHi = (uint32_t)(1024 >> 4) | (1u << 14) | (2u << 29);  // the upper half of both descriptors
      const int t = warp - 14;
      const uint32_t scores = tmem + t * kTile, out = tmem + 256 + t * D;
      const uint32_t idesc_s = f16_idesc(kTile, kTile, kB) | (p.negate << 13);
      const uint32_t idesc_o = f16_idesc(kTile, D, kP) | (1u << 16);  // B with the dimensions innermost
      const uint32_t q_lo = (((base + t * kBytes) & 0x3FFFFu) >> 4) | (1u << 16);  // K-major
      const uint32_t k_lo = ((ring & 0x3FFFFu) >> 4) | (1u << 16);
      const uint32_t v_lo = ((ring & 0x3FFFFu) >> 4) | ((uint32_t)(kPanel >> 4) << 16);  // MN-major
      bool ok = true;
      auto wait = [&](int i, uint32_t phase) {
        ok = mbar_wait(bar(i), phase, abort_flag, kErrMma, a.err);
        return ok;
      };
      auto score = [&](int slot, bool last) {
        if (!in_smem(ring + slot * kBytes, kBytes, raw, a.err)) slot = 0;
        in_smem(base + t * kBytes, kBytes, raw, a.err), in_tmem((uint32_t)(t * kTile), kTile, 512, a.err);
#pragma unroll
        for (int k = 0; k < D / 16; ++k) {
          const uint32_t off = (uint32_t)((k >> 2) * kPanel + (k & 3) * 32) >> 4;
          mma_ss(scores, q_lo + off, k_lo + slot * (kBytes >> 4) + off, kDescHi, idesc_s, k > 0);
        }
        tc_commit(bar(kScores + t));
        tc_commit(bar(kEmpty + slot));
        if (last) tc_commit(bar(kQueriesFree + t));
      };
      auto value = [&](int slot, int part, bool add) {  // 96 or 32 keys
        if (!in_smem(ring + slot * kBytes, kBytes, raw, a.err)) slot = 0;
        in_tmem(256u + (uint32_t)(t * D), D, 512, a.err);
#pragma unroll
        for (int k = part ? 6 : 0; k < (part ? 8 : 6); ++k)
          mma_ts(out, scores + 8 * k, v_lo + slot * (kBytes >> 4) + k * (2048 >> 4), kDescHi, idesc_o, add || k > 0);
      };
      RingPos pos;  // of the next tile
      pos.init(0, kSlots);
      uint32_t prob_phase = 0, free_phase = 1, turns = 0;
      for (int u = 0; ok; ++u) {
        if (!wait(kUnit + (u & 1), (uint32_t)(u >> 1) & 1u) || !read_unit(u)) break;
        mbar_arrive(bar(kUnitFree + (u & 1)));
        const int nt = t ? unit.n[1] : unit.n[0];
        if (!wait(kQueries + t, (uint32_t)u & 1u)) break;
        if (nt == 0) mbar_arrive(bar(kQueriesFree + t));
        if (most == 0) continue;
        if (!wait(kFull + pos.slot, pos.phase)) break;
        tc_fence_after();
        if (nt > 0) score(pos.slot, nt == 1); else mbar_arrive(bar(kEmpty + pos.slot));
        pos.step(1, kSlots);
        for (int j = 0; j < most; ++j, ++turns) {
          const int sv = pos.slot;
          const uint32_t pv = pos.phase;
          pos.step(1, kSlots);
          const int sk = pos.slot;
          const uint32_t pk = pos.phase;
          if (j + 1 < most) pos.step(1, kSlots);
          const bool more = j + 1 < nt;
          // the tiles take turns, so that one's products run while the other's
          // softmax does: in step they would wait for the tensor cores together
          if (!wait(kFull + sv, pv)) break;
          if (j + 1 < most && !wait(kFull + sk, pk)) break;
          if (j == 0 && nt > 0 && !wait(kOutFree + t, free_phase)) break;  // O of the unit before
          if ((t || turns) && !wait(kTurn + t, (t ? turns : turns - 1) & 1u)) break;
          if (j < nt && !wait(kProbs + t, prob_phase)) break;
          if (j < nt) {
            tc_fence_after();
            value(sv, 0, j > 0);
            if (!wait(kProbs + 2 + t, prob_phase)) break;
            prob_phase ^= 1u;
            tc_fence_after();
            value(sv, 1, true);
            tc_commit(bar(kEmpty + sv));
            if (more) score(sk, j + 2 == nt); else tc_commit(bar(kOut + t));
          } else {
            mbar_arrive(bar(kEmpty + sv));  // a tile that only the other rows need
          }
          mbar_arrive(bar(kTurn + 1 - t));
          if (!more && j + 1 < most) mbar_arrive(bar(kEmpty + sk));
        }
        if (nt > 0) free_phase ^= 1u;
      }
      if (!ok) {
        // no product may run past the release of the tensor memory
        tc_commit(bar(kDrain + t));
        mbar_drain(bar(kDrain + t), 0u, a.err);
      }
    }
  }
  tc_fence_before();
  __syncthreads();
  if (warp == 12) {
    tc_fence_after();
    tmem_dealloc(tmem, 512);
  }
}

// Joins the parts of split units: a warp for 32 rows (a lane each) and 32
// dimensions, blockIdx.x the place of a first part and its warp. All places
// are looked at; those that hold no first part end at once. A count of parts
// beyond the places and a row beyond the output (a flag area that was not
// zero) are recorded and touch nothing.
template <bool kB, int D>
__global__ void __launch_bounds__(D) attn_join_kernel(const PromptArgs p) {
  allow_dependent_launch();
  grid_dependency_wait();
  const int lane = threadIdx.x & 31, d0 = threadIdx.x & ~31;
  const float* first = p.partial + (size_t)blockIdx.x * kPartFloats<D>;
  constexpr size_t kNext = (size_t)8 * kPartFloats<D>;
  const int parts = *ld_at(p.joins + blockIdx.x, p.joins, (kFlagBytes - kJoinsAt) / sizeof(int), p.a.err);
  if (parts == 0) return;
  __syncthreads();  // all have read it
  if (threadIdx.x == 0) p.joins[blockIdx.x] = 0;
  const int places = (int)gridDim.x / 8, place = (int)blockIdx.x / 8;
  const int to = reinterpret_cast<const int*>(first)[32 * (D + 2) + lane];
  if (parts < 2 || parts > places - place || to >= p.a.rows * p.a.heads) {
    atomicOr(p.a.err, kErrWorkspace);
    return;
  }
  float m = -INFINITY, l = 0.f;
  float o[32];
#pragma unroll
  for (int i = 0; i < 32; ++i) o[i] = 0.f;
#pragma unroll 2
  for (int i = 0; i < parts; ++i) {
    const float* from = ld_at(first + i * kNext, p.partial, p.partial_floats - kPartFloats<D> + 1, p.a.err);
    const float mi = from[32 * D + lane], li = from[32 * (D + 1) + lane];
    float4 x[8];
#pragma unroll
    for (int k = 0; k < 8; ++k) x[k] = reinterpret_cast<const float4*>(from)[(d0 / 4 + k) * 32 + lane];
    if (li != 0.f) {  // (a part that a row sees no key of holds no O; one with a NaN sum does)
      const float top = fmaxf(m, mi), old = ex2(m - top), f = ex2(mi - top);
      m = top;
      l = l * old + li * f;
#pragma unroll
      for (int k = 0; k < 8; ++k) {
        o[4 * k] = fmaf(x[k].x, f, o[4 * k] * old);
        o[4 * k + 1] = fmaf(x[k].y, f, o[4 * k + 1] * old);
        o[4 * k + 2] = fmaf(x[k].z, f, o[4 * k + 2] * old);
        o[4 * k + 3] = fmaf(x[k].w, f, o[4 * k + 3] * old);
      }
    }
  }
  if (to < 0) return;
  const int head = to % p.a.heads / p.group;
  const float inv = l == 0.f ? 0.f : (p.a.cache.v_scale ? *ld_at(p.a.cache.v_scale + head, p.a.cache.v_scale, (size_t)p.a.cache.kv_heads, p.a.err) : 1.f) / l;
  uint16_t* dst = p.a.out + (size_t)to * D + d0;
  if (!in_buf(dst + 24, p.a.out, (size_t)p.a.rows * p.a.heads * D - 7, p.a.err)) return;
#pragma unroll
  for (int i = 0; i < 32; i += 8)
    *reinterpret_cast<uint4*>(dst + i) =
        make_uint4(pack16<kB>(o[i] * inv, o[i + 1] * inv), pack16<kB>(o[i + 2] * inv, o[i + 3] * inv),
                   pack16<kB>(o[i + 4] * inv, o[i + 5] * inv), pack16<kB>(o[i + 6] * inv, o[i + 7] * inv));
  if (p.a.lse && d0 == 0) p.a.lse[to] = l == 0.f ? -INFINITY : m * kLn2 + logf(l);
}

// Tensor map of a row-major array: dims and box innermost first, strides of
// the outer dimensions in bytes. Encoded by each call: half a microsecond, and
// nothing is kept by a buffer's address.
bool encode_tiles(CUtensorMap* out, const void* ptr, CUtensorMapDataType type, int rank, const cuuint64_t (&dims)[3],
                  const cuuint64_t (&strides)[2], const cuuint32_t (&box)[3], CUtensorMapSwizzle swizzle) {
  static const PFN_cuTensorMapEncodeTiled_v12000 encode = []() -> PFN_cuTensorMapEncodeTiled_v12000 {
    void* fn = nullptr;
    cudaDriverEntryPointQueryResult found;
    if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &fn, 12000, cudaEnableDefault, &found) != cudaSuccess ||
        found != cudaDriverEntryPointSuccess)
      return nullptr;
    return reinterpret_cast<PFN_cuTensorMapEncodeTiled_v12000>(fn);
  }();
  const cuuint32_t steps[3] = {1, 1, 1};
  return encode && encode(out, type, (cuuint32_t)rank, const_cast<void*>(ptr), dims, strides, box, steps,
                          CU_TENSOR_MAP_INTERLEAVE_NONE, swizzle, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                          CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

template <bool kB, bool k8, int D>
cudaError_t launch(PromptArgs p, unsigned blocks, cudaStream_t stream) {
  // the caches as rows of D values, copied by up to 128 rows of a page, in
  // panels of 64 dimensions or whole rows of codes (row numbers are 32-bit
  // coordinates: the cache's rows are below 2^31)
  CUtensorMap map_k = {}, map_v = {}, map_q = {};
  const long long rows = ((long long)p.a.cache.pages * p.a.cache.kv_heads) << p.a.cache.page_shift;
  const auto type16 = kB ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_FLOAT16;
  const auto type = k8 ? CU_TENSOR_MAP_DATA_TYPE_UINT8 : type16;
  const auto swizzle = k8 ? CU_TENSOR_MAP_SWIZZLE_NONE : CU_TENSOR_MAP_SWIZZLE_128B;
  const cuuint64_t dims[3] = {D, (cuuint64_t)rows, 1}, strides[2] = {D * (k8 ? 1 : 2), 0};
  const cuuint32_t box[3] = {k8 ? D : 64, 1u << (p.a.cache.page_shift < 7 ? p.a.cache.page_shift : 7), 1};
  if (!encode_tiles(&map_k, p.a.cache.k, type, 2, dims, strides, box, swizzle) ||
      !encode_tiles(&map_v, p.a.cache.v, type, 2, dims, strides, box, swizzle))
    return cudaErrorInvalidValue;
  // the queries as [tokens][heads][D], where a tile of 128 rows is whole
  // tokens of a key/value head's group
  p.q_tiled = kTile % p.group == 0;
  if (p.q_tiled) {
    const cuuint64_t q_dims[3] = {D, (cuuint64_t)p.a.heads, (cuuint64_t)p.a.rows};
    const cuuint64_t q_strides[2] = {D * 2, (cuuint64_t)p.a.ldq * 2};
    const cuuint32_t q_box[3] = {64, (cuuint32_t)p.group, (cuuint32_t)(kTile / p.group)};
    if (!encode_tiles(&map_q, p.a.q, type16, 3, q_dims, q_strides, q_box, CU_TENSOR_MAP_SWIZZLE_128B)) return cudaErrorInvalidValue;
  }
  auto kern = attn_prompt_kernel<kB, k8, D>;
  cudaError_t e = set_max_smem_once(reinterpret_cast<const void*>(kern), kSmem<D>);
  if (e != cudaSuccess) return e;
  e = launch_pdl(kern, dim3(blocks), dim3(kThreads), kSmem<D>, stream, p, map_k, map_v, map_q);
  if (e != cudaSuccess || p.most_parts < 2) return e;
  return launch_pdl(attn_join_kernel<kB, D>, dim3(blocks * 8), dim3(D), 0, stream, p);
}

// Whether the units can be fewer than the blocks.
bool may_split(int tokens, int group, int kv_heads, int sms) {
  return ((long long)tokens * group + 2 * kTile - 1) / (2 * kTile) * kv_heads < sms;
}

}  // namespace

size_t attn_prompt_workspace_bytes(int tokens, int group, int kv_heads, int head_dim, int sms) {
  return kFlagBytes + (may_split(tokens, group, kv_heads, sms) ? (size_t)sms * 8 * 32 * (head_dim + 3) * sizeof(float) : 0);
}

cudaError_t launch_attn_prompt(const AttnArgs& args, int head_dim, bool bf16, bool e4m3, void* workspace, int sms,
                               cudaStream_t stream) {
  if (args.rows == 0 || args.batch == 0) return cudaSuccess;
  PromptArgs p;
  p.a = args;
  cudaError_t e = device_error_word(&p.a.err);
  if (e != cudaSuccess) return e;
  p.group = args.heads / args.cache.kv_heads;
  // the scores' maximum is taken before the scale, so it has to be positive:
  // a negative scale negates the product, and a scale of zero becomes one too
  // small to tell from it
  p.mult = fmaxf(fabsf(args.scale) * kLog2e, 1e-37f);
  p.negate = args.scale < 0.f;
  p.queue = static_cast<int*>(workspace);
  p.partial = reinterpret_cast<float*>(static_cast<uint8_t*>(workspace) + kFlagBytes);
  p.joins = reinterpret_cast<int*>(static_cast<uint8_t*>(workspace) + kJoinsAt);
  p.partial_floats = (attn_prompt_workspace_bytes(args.rows, p.group, args.cache.kv_heads, head_dim, sms) - kFlagBytes) / sizeof(float);
  // a block per SM, or as many as there can be units (whole ones of all rows,
  // and a ragged one per sequence) where none is long enough for two parts
  const long long units = ((long long)args.rows * p.group / (2 * kTile) + args.batch) * args.cache.kv_heads;
  const long long tiles = (((long long)args.max_pages << args.cache.page_shift) + kTile - 1) / kTile;
  p.most_parts = 1;
  if (may_split(args.rows, p.group, args.cache.kv_heads, sms) && tiles >= 2 * kLeast)
    p.most_parts = (int)(tiles / kLeast < sms ? tiles / kLeast : sms);
  const unsigned blocks = units < sms && p.most_parts < 2 ? (unsigned)units : (unsigned)sms;
  switch ((bf16 ? 4 : 0) | (e4m3 ? 2 : 0) | (head_dim == 128 ? 1 : 0)) {
    case 0: return launch<false, false, 64>(p, blocks, stream);
    case 1: return launch<false, false, 128>(p, blocks, stream);
    case 2: return launch<false, true, 64>(p, blocks, stream);
    case 3: return launch<false, true, 128>(p, blocks, stream);
    case 4: return launch<true, false, 64>(p, blocks, stream);
    case 5: return launch<true, false, 128>(p, blocks, stream);
    case 6: return launch<true, true, 64>(p, blocks, stream);
    default: return launch<true, true, 128>(p, blocks, stream);
  }
}

}  // namespace w4a16
