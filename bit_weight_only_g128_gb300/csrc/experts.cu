// W4A16 products grouped by expert, for few rows per expert, and the weighted
// sum over a token's experts.
//
// Choice f of expert e: Y[f][n] = sum_k A[f or f / top][k] (q - z) s [e][k][n],
// with the gate/up epilogue silu(gate) * up of columns [gate | up], or summed
// over a token's choices with their weights.
//
// Every expert that has rows streams its packed weights once per 16 rows, so
// the bound is HBM bytes, and for a token or two the chain offsets - rows -
// activations and weights - sums. An item of work is up to 16 rows of one expert
// times 128 / KS columns; a block's 8 warps take a strip of 16 columns each and
// one of KS parts of K, so that few rows still spread over all SMs. The blocks
// are persistent, two per SM, and take the items in turn; weights (three units
// of four atoms ahead, each warp its own), scales and activations (two units
// ahead, gathered by row) stream into shared memory by asynchronous copies that
// run on across the items. The codes enter
// mma.sync m16n8k16 as exact 16-bit numbers without a multiplication: fp16
// takes q masked in place as the subnormal q 2^-24 (the odd pairs one nibble
// higher, summed apart and divided by 16), bf16 takes (128 + q) 2^-12 put
// together by byte permutes; the zero point, in the same form, is subtracted
// exactly. Each group's fp32 sum is multiplied by its scale (and 2^24 or 2^12). So
// the weights are (q - z) s unrounded, the sums fp32, and the result is rounded
// once. (Zero points multiplied and subtracted in the sums would make NaN of an
// infinite activation, and of a bf16 one from 2^121 on, where q - z times it is
// not: inf - inf; the four MMAs that took a pair of atoms' place of 32
// subtractions were no faster: gate and up of 1 token 8.2 us against 7.6, of 16
// 37.3 against 36.0. The 2^-12 keeps a group's sum of up to 273 products of any
// finite bf16 activations finite, below 2^128 15 273 2^-12, before its scale.)
//
// Combined, each choice's product goes to the workspace in fp32, and a second
// kernel adds a token's rows, multiplied by their weights, in the order of its
// choices: no atomics, the same result every time.
//
// Measured (us a call, bytes of weights and rows a second): gate and up of 2048 x
// 2048 over 64 experts, top 8, 1 token 7.6 (2.3 TB/s), 16 tokens, bf16, 36 (3.4);
// of 4096 x 22016 over 8, top 2, 32 tokens 108-114 (3.4, half of the copy rate, 0.61
// instructions a cycle and scheduler: sixteen warps on an SM, which the registers of
// the sums and codes allow, cannot hide all the latency of shared memory and MMAs);
// down of 1024 x 2048 over 64, 1 token 8.0-8.6, 100 tokens 41 (0.53 a cycle).
#include <cuda_bf16.h>

#include <cmath>
#include <type_traits>

#include "experts.cuh"

namespace w4a16 {
namespace {

constexpr int kThreads = 256;
constexpr int kWarps = 8;
constexpr int kRows = 16;      // most rows of an item
constexpr int kUnit = 4;       // atoms of a step
constexpr int kWeightSlots = 4, kRowSlots = 3;  // units in shared memory: weights, activations
constexpr int kUnitBytes = kUnit * kAtomWords * 4;         // a warp's codes of a unit
constexpr int kSlotBytes = kUnitBytes + 2 * 32 * 4;        // with its scales and zero points
constexpr int kRowBytes = kUnit * 128 + 64;  // of a unit's activations: neighbouring rows in opposite halves of the banks
constexpr int kItems = 8;      // items known at a time
constexpr int kMostExperts = 512;
constexpr uint32_t kFull = 0xffffffffu;

struct DecodeParams {
  ExpertArgs a;
  float* D;      // combined: [choices][N]
  int blocks;    // column blocks
  int tile;      // rows of an item at most: 8 or 16, and no more than T
};

__device__ __forceinline__ void copies_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void copies_wait() { asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory"); }

// The bf16 2^-5 = 128 * 2^-12, whose low 4 of 7 fraction bits count 2^-12: the
// byte above a code's (the byte 0x0q), and two with codes of zero.
constexpr uint32_t kBf16Code = 0x3d3d3d3du, kBf16Zero = 0x3d003d00u;

// A zero point in the codes' form: lo for pairs 0 and 1, hi for 2 and 3 (bf16:
// one form for all).
template <bool kB>
struct Zero {
  uint32_t lo, hi;
  __device__ __forceinline__ explicit Zero(uint32_t z) {
    if (kB) {
      lo = hi = kBf16Zero | z | (z << 16);
    } else {
      lo = z | (z << 16);
      hi = lo << 4;
    }
  }
};

// The four pairs of a word minus the zero point: (k 0, 1), (2, 3), (4, 5),
// (6, 7); exact. fp16: (q - z) 2^-24 in the first two, 16 times that in the
// others; bf16: (q - z) 2^-12.
template <bool kB>
__device__ __forceinline__ void codes(uint32_t w, const Zero<kB>& z, uint32_t (&c)[4]) {
  if (kB) {
    const uint32_t t = w & 0x0F0F0F0Fu, u = (w >> 4) & 0x0F0F0F0Fu;
    c[0] = __byte_perm(t, kBf16Code, 0x4240);
    c[1] = __byte_perm(t, kBf16Code, 0x4341);
    c[2] = __byte_perm(u, kBf16Code, 0x4240);
    c[3] = __byte_perm(u, kBf16Code, 0x4341);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const __nv_bfloat162 d = __hsub2(*reinterpret_cast<const __nv_bfloat162*>(&c[i]), *reinterpret_cast<const __nv_bfloat162*>(&z.lo));
      c[i] = *reinterpret_cast<const uint32_t*>(&d);
    }
  } else {
    const uint32_t w8 = w >> 8;
    c[0] = hsub2_rn(w & 0x000F000Fu, z.lo);
    c[1] = hsub2_rn(w8 & 0x000F000Fu, z.lo);
    c[2] = hsub2_rn(w & 0x00F000F0u, z.hi);
    c[3] = hsub2_rn(w8 & 0x00F000F0u, z.hi);
  }
}

// An item: rows of expert e (E: of none, whose results are zeros) times a
// block of columns.
struct Item {
  int e, n, col;
  int of[kRows], src[kRows];  // choice and row of A
};

// KS: parts of K. kPairs: groups of 128 k, two atoms, of which a unit has two
// and a part a whole number; else any.
template <bool kB, int KS, bool kPairs>
__global__ void __launch_bounds__(kThreads, 2) experts_decode_kernel(const DecodeParams p) {
  constexpr int S = kWarps / KS;        // strips of an item
  constexpr int kCols = S * kStripCols;
  constexpr int kRed = kCols + 4;       // floats of a row of partial sums
  extern __shared__ __align__(128) uint8_t dynamic[];
  __shared__ float red[KS][kRows][kRed];
  __shared__ Item items[kItems];
  __shared__ int offs[kMostExperts + 2], firsts[kMostExperts + 2];  // experts' offsets and first row tiles
  const ExpertArgs& a = p.a;
  const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
  const uint32_t dyn = (uint32_t)__cvta_generic_to_shared(dynamic);
  const uint32_t weights = dyn + (uint32_t)warp * kWeightSlots * kSlotBytes;  // this warp's units
  const uint32_t rows = dyn + kWarps * kWeightSlots * kSlotBytes;             // the block's activations
  const uint32_t row_slot = (uint32_t)(KS * p.tile) * kRowBytes;
  const int part = warp / S, w = warp % S;  // this warp's part of K, and its strip of an item
  const int natoms = a.K / kAtomK, G = a.K / a.group, apg = a.group / kAtomK;
  // first atom of a part of K
  auto part_begin = [&](int k) { return kPairs ? natoms / 2 * k / KS * 2 : natoms * k / KS; };
  const int begin = part_begin(part), end = part_begin(part + 1);  // this warp's atoms
  const int longest = kPairs ? (natoms / 2 + KS - 1) / KS * 2 : (natoms + KS - 1) / KS;
  const int units = (longest + kUnit - 1) / kUnit;                       // steps of an item
  const int half = a.N / 2, width = a.silu ? half : a.N;                 // of a result's row
  const int cols = a.silu ? kCols / 2 : kCols;                           // of an item's results
  allow_dependent_launch();
  grid_dependency_wait();

  // the row tiles: of one token a choice each, else from the offsets
  int tiles = a.top;
  if (a.T > 1) {
    if (warp == 0) {
      // offsets that never decrease (recorded where they do), the last that of
      // the choices' end; the prefix sums of the tiles
      int top = 0, sum = 0;
      for (int e0 = 0; e0 <= a.E + 1; e0 += 32) {
        const int e = e0 + lane;
        const int v = e <= a.E ? offset_of(a, e) : choices(a);
        int m = max(v, top);
#pragma unroll
        for (int d = 1; d < 32; d <<= 1) {
          const int u = __shfl_up_sync(kFull, m, d);
          if (lane >= d) m = max(m, u);
        }
        if (e <= a.E && m != v) atomicOr(a.err, kErrRange);
        // the tiles of expert e - 1, which ends here
        int before = __shfl_up_sync(kFull, m, 1);
        if (lane == 0) before = top;
        int s = e > 0 && e <= a.E + 1 ? (m - before + p.tile - 1) / p.tile : 0;
#pragma unroll
        for (int d = 1; d < 32; d <<= 1) {
          const int u = __shfl_up_sync(kFull, s, d);
          if (lane >= d) s += u;
        }
        if (e <= a.E + 1) {
          offs[e] = m;
          firsts[e] = sum + s;
        }
        sum += __shfl_sync(kFull, s, 31);
        top = __shfl_sync(kFull, m, 31);
      }
    }
    __syncthreads();
    tiles = firsts[a.E + 1];
  }
  // (below 2^30: a full item has 256 results or more, of which 280 GB hold 2^37, and
  // of others each expert has one per 32 columns, E * N / 32 below 2^26; divisions in 64
  // bits cost one token 0.2 us)
  const uint32_t all = (uint32_t)tiles * (uint32_t)p.blocks;
  // this block's items: blockIdx.x, blockIdx.x + gridDim.x, ...
  const int count = blockIdx.x < all ? (int)((all - 1 - blockIdx.x) / gridDim.x) + 1 : 0;
  // item i of the block, written down by a warp
  auto describe = [&](int i) {
    if (i >= count) return;
    const uint32_t at = blockIdx.x + (uint32_t)i * gridDim.x;
    // (row tiles first: those of one expert read the same weights)
    const int col = (int)(at / (uint32_t)tiles), tile = (int)(at % (uint32_t)tiles);
    int e, first, n = 1;
    if (a.T == 1) {
      first = tile;
      e = *ld_at(a.experts + tile, a.experts, (size_t)choices(a), a.err);
      if (e >= a.E) {
        if (lane == 0) atomicOr(a.err, kErrRange);
        e = -1;
      }
      if (e < 0) e = a.E;
    } else {
      int lo = 0, hi = a.E + 1;  // the last expert whose first tile is not behind
      while (hi - lo > 1) {
        const int mid = (lo + hi) / 2;
        if (firsts[mid] <= tile) lo = mid;
        else hi = mid;
      }
      e = lo;
      first = offs[e] + (tile - firsts[e]) * p.tile;
      n = min(p.tile, offs[e + 1] - first);
    }
    Item& it = items[i % kItems];
    if (lane == 0) it.e = e, it.n = n, it.col = col;
    if (lane < kRows) {
      int f = -1;
      if (lane < n) f = a.T == 1 ? first : choice_of(a, first + lane);
      it.of[lane] = f;
      it.src[lane] = f < 0 ? 0 : a.per_choice ? f : f / a.top;
    }
  };
  if (warp < kWeightSlots) describe(warp);
  __syncthreads();

  // The stream of weights of this warp: the next unit to copy, this lane's first
  // word of it (null: no strip), and with kPairs its word of scales or zero points.
  // (with silu an item's first strips are gate columns, the rest the up columns
  // of the same results)
  int wi = 0, wu = 0, wslot = 0, strip = 0;
  const uint4* codes_from = nullptr;
  const uint32_t* meta_from = nullptr;
  const uint4* const wq = reinterpret_cast<const uint4*>(a.Wq);
  const uint32_t* const sp = reinterpret_cast<const uint32_t*>(a.Sp);
  const size_t all_codes = (size_t)a.E * a.N * a.K / 32, all_scales = (size_t)a.E * a.N * G / 2;
  auto enter = [&]() {
    codes_from = nullptr;
    if (wi >= count) return;
    const Item& it = items[wi % kItems];
    if (it.e >= a.E) return;
    int s = it.col * S + w;
    bool live = s < a.N / kStripCols;
    if (a.silu) {
      s = it.col * (S / 2) + w % (S / 2);
      live = s < half / kStripCols;
      if (w >= S / 2) s += half / kStripCols;
    }
    if (!live) return;
    strip = it.e * (a.N / kStripCols) + s;
    codes_from = wq + ((size_t)strip * natoms + begin) * 32 + lane;
    const size_t at = (size_t)strip * G + begin / 2;
    if (kPairs) meta_from = lane < 16 ? sp + at * 8 + lane : a.Zp + at * 2 + lane - 16;
  };
  auto copy_weights = [&]() {
    const int n = min(kUnit, end - begin - wu * kUnit);
    if (codes_from && n > 0) {
      const uint32_t to = weights + (uint32_t)wslot * kSlotBytes;
#pragma unroll
      for (int j = 0; j < kUnit; ++j)
        if (j < n && in_smem(to + 512u * j + 16u * lane, 16, dyn, a.err))
          copy16(to + 512u * j + 16u * lane, ld_at(codes_from + 32 * j, wq, all_codes, a.err));
      codes_from += 32 * kUnit;
      if (kPairs) {
        // lane 8 i + c: the scales of columns c and c + 8 of the unit's group i;
        // lane 16 + 2 i + h: the zero points of columns 4 h .. 4 h + 3, each with
        // its column + 8
        if (lane < 16 ? lane < 4 * n : lane < 16 + n)
          copy4(to + kUnitBytes + 4u * lane,
                lane < 16 ? ld_at(meta_from, sp, all_scales, a.err) : ld_at(meta_from, a.Zp, all_scales / 4, a.err));
        meta_from += lane < 16 ? 16 : 4;
      } else {
        // lane 8 i + c: the scales of columns c and c + 8 of the unit's i-th
        // group, and the word of zero points that c's is in
        const int a0 = begin + wu * kUnit, g = a0 / apg + lane / 8;
        if (g <= (a0 + n - 1) / apg) {
          const size_t at = (size_t)strip * G + g;
          copy4(to + kUnitBytes + 4u * lane, ld_at(sp + at * 8 + lane % 8, sp, all_scales, a.err));
          copy4(to + kUnitBytes + 128u + 4u * lane, ld_at(a.Zp + at * 2 + lane % 8 / 4, a.Zp, all_scales / 4, a.err));
        }
      }
    }
    wslot = wslot + 1 == kWeightSlots ? 0 : wslot + 1;
    if (++wu == units && wi < count) {
      wu = 0;
      ++wi;
      // the item three on is written down now, by one warp
      if (wi % kWarps == warp) describe(wi + kWeightSlots - 1);
      enter();
    }
  };
  // The block's stream of activations: a unit of every part. This warp copies
  // the rows (warp + 8 m) / KS of part warp % KS, a lane 16 bytes of each; src:
  // which rows of A those are for the item that the stream is in.
  constexpr int kPasses = kRows * KS / kWarps;
  int ri = 0, ru = 0, rslot = 0, rn = 0;  // rn: the item's rows
  int src[kPasses];
  const int rbegin = part_begin(warp % KS), rend = part_begin(warp % KS + 1);
  auto enter_rows = [&]() {
    rn = 0;
    if (ri >= count) return;
    const Item& it = items[ri % kItems];
    if (it.e < a.E) rn = it.n;
#pragma unroll
    for (int m = 0; m < kPasses; ++m) src[m] = it.src[(warp + kWarps * m) / KS];
  };
  auto copy_rows = [&]() {
    const int k0 = rbegin + ru * kUnit + lane / 8;  // the lane's atom
    if (k0 < rend) {
      const uint32_t to = rows + (uint32_t)rslot * row_slot +
                          (uint32_t)(warp % KS * p.tile + warp / KS) * kRowBytes + 16u * lane;
      const uint16_t* from = a.A + k0 * kAtomK + lane % 8 * 8;
#pragma unroll
      for (int m = 0; m < kPasses; ++m) {
        if ((warp + kWarps * m) / KS >= rn) break;
        const uint32_t at = to + (uint32_t)(m * (kWarps / KS)) * kRowBytes;
        if (in_smem(at, 16, dyn, a.err))
          copy16(at, ld_at(from + (uint64_t)(uint32_t)src[m] * (uint32_t)a.K, a.A, a_elements(a) - 7, a.err));
      }
    }
    rslot = rslot + 1 == kRowSlots ? 0 : rslot + 1;
    if (++ru == units) {
      ru = 0;
      ++ri;
      enter_rows();
    }
  };

  float out[2][4] = {};
  const float scale = kB ? 4096.f : 16777216.f;  // of the codes' form
  auto scales = [&](uint32_t sw, float& s0, float& s1) {
    s0 = value16<false>(sw & 0xffffu) * scale, s1 = value16<false>(sw >> 16) * scale;
  };
  // out += a unit's products: MT octets of rows
  auto multiply_pairs = [&](auto octets, uint32_t wt, uint32_t act, int i0, int i1) {  // the pairs i0 .. i1
    constexpr int MT = decltype(octets)::value;
#pragma unroll
    for (int i = i0; i < i1; ++i) {
      uint32_t sw, zw;
      asm volatile("ld.shared.u32 %0, [%1];" : "=r"(sw) : "r"(wt + kUnitBytes + (uint32_t)(8 * i + lane / 4) * 4u) : "memory");
      asm volatile("ld.shared.u32 %0, [%1];" : "=r"(zw) : "r"(wt + kUnitBytes + 64u + (uint32_t)(2 * i + lane / 16) * 4u) : "memory");
      const uint32_t zz = zw >> (lane / 4 % 4 * 8);
      const Zero<kB> z0(zz & 15u), z1((zz >> 4) & 15u);
      float lo[MT][4], hi[MT][4];
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        const uint4 v = tc::lds128(wt + 512u * (2 * i + j) + 16u * lane);
        const uint32_t wd[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
        for (int s = 0; s < 2; ++s) {
          uint32_t c0[4], c1[4];
          codes<kB>(wd[2 * s], z0, c0);
          codes<kB>(wd[2 * s + 1], z1, c1);
#pragma unroll
          for (int m = 0; m < MT; ++m) {
            const uint4 b = tc::lds128(act + m * 8 * kRowBytes + (2 * i + j) * 128 + s * 64);
            float(&second)[4] = kB ? lo[m] : hi[m];
            if (j == 0 && s == 0) {
              mma_first<kB>(lo[m], c0[0], c1[0], c0[1], c1[1], b.x, b.y);
              if (kB)
                mma_acc<kB>(second, c0[2], c1[2], c0[3], c1[3], b.z, b.w);
              else
                mma_first<kB>(second, c0[2], c1[2], c0[3], c1[3], b.z, b.w);
            } else {
              mma_acc<kB>(lo[m], c0[0], c1[0], c0[1], c1[1], b.x, b.y);
              mma_acc<kB>(second, c0[2], c1[2], c0[3], c1[3], b.z, b.w);
            }
          }
        }
      }
      float s0, s1;
      scales(sw, s0, s1);
#pragma unroll
      for (int m = 0; m < MT; ++m)
#pragma unroll
        for (int k = 0; k < 4; ++k)
          out[m][k] = fmaf(kB ? lo[m][k] : fmaf(hi[m][k], 0.0625f, lo[m][k]), k < 2 ? s0 : s1, out[m][k]);
    }
  };
  auto multiply_any = [&](auto octets, uint32_t wt, uint32_t act, int a0, int n) {
    constexpr int MT = decltype(octets)::value;
    float lo[MT][4] = {}, hi[MT][4] = {};
    int left = apg - a0 % apg, g = 0;  // atoms left of the group, group of the unit
    float s0 = 0.f, s1 = 0.f;
    uint32_t zz = 0;
    auto group = [&]() {
      const uint32_t at = wt + kUnitBytes + (uint32_t)(8 * g + lane / 4) * 4u;
      uint32_t sw, zw;
      asm volatile("ld.shared.u32 %0, [%1];" : "=r"(sw) : "r"(at) : "memory");
      asm volatile("ld.shared.u32 %0, [%1];" : "=r"(zw) : "r"(at + 128u) : "memory");
      zz = zw >> (lane / 4 % 4 * 8);
      scales(sw, s0, s1);
    };
    group();
#pragma unroll
    for (int j = 0; j < kUnit; ++j) {
      if (j >= n) break;
      const uint4 v = tc::lds128(wt + 512u * j + 16u * lane);
      const Zero<kB> z0(zz & 15u), z1((zz >> 4) & 15u);
      const uint32_t wd[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
      for (int s = 0; s < 2; ++s) {
        uint32_t c0[4], c1[4];
        codes<kB>(wd[2 * s], z0, c0);
        codes<kB>(wd[2 * s + 1], z1, c1);
#pragma unroll
        for (int m = 0; m < MT; ++m) {
          const uint4 b = tc::lds128(act + m * 8 * kRowBytes + j * 128 + s * 64);
          mma_acc<kB>(lo[m], c0[0], c1[0], c0[1], c1[1], b.x, b.y);
          mma_acc<kB>(kB ? lo[m] : hi[m], c0[2], c1[2], c0[3], c1[3], b.z, b.w);
        }
      }
      if (--left == 0 || j + 1 == n) {
#pragma unroll
        for (int m = 0; m < MT; ++m)
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            out[m][i] = fmaf(kB ? lo[m][i] : fmaf(hi[m][i], 0.0625f, lo[m][i]), i < 2 ? s0 : s1, out[m][i]);
            lo[m][i] = hi[m][i] = 0.f;
          }
        if (left == 0 && j + 1 < n) {
          left = apg;
          ++g;
          group();
        }
      }
    }
  };
  auto multiply = [&](auto octets, uint32_t wt, uint32_t act, int a0, int n) {
    if constexpr (kPairs) {
      if (n == kUnit) multiply_pairs(octets, wt, act, 0, kUnit / 2);  // (a constant number, without branches)
      else multiply_pairs(octets, wt, act, 0, 1);
    }
    else multiply_any(octets, wt, act, a0, n);
  };

  // every step commits one group of copies: weights of unit s + 3, activations
  // of unit s + 2
  enter();
  enter_rows();
  for (int u = 0; u < kWeightSlots - 1; ++u) {
    copy_weights();
    if (u > 0) copy_rows();
    copies_commit();
    // (items that the stream has entered are written down for the next one)
    __syncthreads();
  }
  int cslot = 0, aslot = 0;
  for (int i = 0; i < count; ++i) {
    const Item& it = items[i % kItems];
    for (int u = 0; u < units; ++u) {
      copies_wait<kWeightSlots - 3>();  // this step's weights and activations
      __syncthreads();
      copy_weights();
      copy_rows();
      copies_commit();
      const int a0 = begin + u * kUnit, n = min(kUnit, end - a0);
      if (n > 0 && it.e < a.E) {
        const uint32_t wt = weights + (uint32_t)cslot * kSlotBytes;
        const uint32_t act = rows + (uint32_t)aslot * row_slot + (uint32_t)(part * p.tile + lane / 4) * kRowBytes + lane % 4 * 16u;
        if (it.n <= 8)
          multiply(std::integral_constant<int, 1>(), wt, act, a0, n);
        else
          multiply(std::integral_constant<int, 2>(), wt, act, a0, n);
      }
      cslot = cslot + 1 == kWeightSlots ? 0 : cslot + 1;
      aslot = aslot + 1 == kRowSlots ? 0 : aslot + 1;
    }
    // sums by row: lane (g, t) holds columns g, g + 8 of rows 2t, 2t + 1
#pragma unroll
    for (int m = 0; m < 2; ++m)
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        red[part][m * 8 + (lane % 4) * 2 + (j & 1)][w * kStripCols + lane / 4 + (j & 2) * 4] = out[m][j];
        out[m][j] = 0.f;
      }
    __syncthreads();
    const int n0 = it.col * cols;
    for (int k = threadIdx.x; k < it.n * (cols / 2); k += kThreads) {
      const int r = k / (cols / 2), c = k % (cols / 2) * 2, n = n0 + c;
      if (it.of[r] < 0 || n >= width || (a.combine && it.e >= a.E)) continue;
      float v[2] = {0.f, 0.f}, g[2] = {0.f, 0.f};
#pragma unroll
      for (int q = 0; q < KS; ++q)
#pragma unroll
        for (int j = 0; j < 2; ++j) {
          v[j] += red[q][r][c + j];
          if (a.silu) g[j] += red[q][r][kCols / 2 + c + j];
        }
      if (it.e >= a.E) v[0] = v[1] = g[0] = g[1] = 0.f;
      const size_t at = (size_t)it.of[r] * width + n, everything = (size_t)choices(a) * width - 1;
      if (a.combine) {
        float* d = p.D + at;
        if (in_buf(d, p.D, everything, a.err)) *reinterpret_cast<float2*>(d) = make_float2(v[0], v[1]);
      } else {
        if (a.silu) v[0] = silu_times(v[0], g[0]), v[1] = silu_times(v[1], g[1]);
        uint16_t* y = a.Y + at;
        if (in_buf(y, a.Y, everything, a.err)) *reinterpret_cast<uint32_t*>(y) = pack16<kB>(v[0], v[1]);
      }
    }
  }
  copies_wait<0>();
}

// Eight columns of a row of products, 16-bit or fp32, as loaded and as values.
struct Eight16 {
  uint4 u;
  __device__ __forceinline__ void load(const uint16_t* p) { u = __ldcs(reinterpret_cast<const uint4*>(p)); }
  template <bool kB>
  __device__ __forceinline__ void values(float (&v)[8]) const {
    const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float2 f = unpack16<kB>(w[i]);
      v[2 * i] = f.x, v[2 * i + 1] = f.y;
    }
  }
};
struct Eight32 {
  float4 a, b;
  __device__ __forceinline__ void load(const float* p) {
    a = __ldcs(reinterpret_cast<const float4*>(p)), b = __ldcs(reinterpret_cast<const float4*>(p) + 1);
  }
  template <bool kB>
  __device__ __forceinline__ void values(float (&v)[8]) const {
    v[0] = a.x, v[1] = a.y, v[2] = a.z, v[3] = a.w, v[4] = b.x, v[5] = b.y, v[6] = b.z, v[7] = b.w;
  }
};

// Y[t] = the weighted sum of the rows of D of token t's choices that have an
// expert, in their order, in fp32. One thread per eight columns; eight choices
// in flight, of 16-bit products four (eight would take the registers of every
// third block: 172 against 164 us with the products of 4099 tokens, top 8, 2048
// columns). Products that are infinite in fp16 are read from `wide`, [choices][N]
// in fp32. Bound: HBM bytes, for a token or two the chain experts - products.
template <bool kB, class T, class Loaded>
__global__ void __launch_bounds__(kThreads) experts_sum_kernel(const ExpertArgs a, const T* D, const float* wide) {
  constexpr int kFlight = sizeof(T) == 2 ? 4 : 8;
  allow_dependent_launch();
  grid_dependency_wait();
  const int vecs = a.N / 8;
  // vector kThreads * block + thread of them all, in 32 bits: vecs blocks are
  // kThreads rows
  const uint32_t in = blockIdx.x % (uint32_t)vecs * kThreads + threadIdx.x;
  const int t = (int)(blockIdx.x / (uint32_t)vecs * kThreads + in / (uint32_t)vecs), n = (int)(in % (uint32_t)vecs) * 8;
  if (t >= a.T) return;
  const size_t f0 = (size_t)t * a.top;
  float sum[8] = {};
  for (int j0 = 0; j0 < a.top; j0 += kFlight) {
    bool live[kFlight];
    float w[kFlight];
    Loaded d[kFlight];
#pragma unroll
    for (int j = 0; j < kFlight; ++j) {
      live[j] = j0 + j < a.top;
      if (live[j]) {
        w[j] = *ld_at(a.weights + f0 + j0 + j, a.weights, (size_t)choices(a), a.err);
        const int e = *ld_at(a.experts + f0 + j0 + j, a.experts, (size_t)choices(a), a.err);
        live[j] = (unsigned)e < (unsigned)a.E;
        if (e >= a.E) atomicOr(a.err, kErrRange);  // (none: the products may have left its row unwritten)
      }
    }
#pragma unroll
    for (int j = 0; j < kFlight; ++j)
      if (live[j]) d[j].load(ld_at(D + (f0 + j0 + j) * a.N + n, D, (size_t)choices(a) * a.N - 7, a.err));
#pragma unroll
    for (int j = 0; j < kFlight; ++j) {
      if (!live[j]) continue;
      float v[8];
      d[j].template values<kB>(v);
#pragma unroll
      for (int k = 0; k < 8; ++k) sum[k] = fmaf(w[j], v[k], sum[k]);
    }
  }
  if constexpr (!kB && sizeof(T) == 2) {
    // an infinite product leaves its sum infinite or NaN: once more, with `wide`
    // (asked of the sums at the end: of every product it cost 1.5 us of 27 at the
    // case above)
    float any = 0.f;
#pragma unroll
    for (int k = 0; k < 8; ++k) any = fmaf(sum[k], 0.f, any);
    if (any != 0.f) {
#pragma unroll 1
      for (int k = 0; k < 8; ++k) {
        float s = 0.f;
#pragma unroll 1
        for (size_t f = f0; f < f0 + a.top; ++f) {
          if ((unsigned)*ld_at(a.experts + f, a.experts, (size_t)choices(a), a.err) >= (unsigned)a.E) continue;
          const size_t at = f * a.N + n + k, all = (size_t)choices(a) * a.N;
          float v = value16<kB>(*ld_at(D + at, D, all, a.err));
          if (isinf(v)) v = *ld_at(wide + at, wide, all, a.err);
          s = fmaf(*ld_at(a.weights + f, a.weights, (size_t)choices(a), a.err), v, s);
        }
#pragma unroll
        for (int i = 0; i < 8; ++i)
          if (i == k) sum[i] = s;
      }
    }
  }
  uint16_t* y = a.Y + (size_t)t * a.N + n;
  if (in_buf(y, a.Y, (size_t)a.T * a.N - 7, a.err))
    *reinterpret_cast<uint4*>(y) = make_uint4(pack16<kB>(sum[0], sum[1]), pack16<kB>(sum[2], sum[3]),
                                              pack16<kB>(sum[4], sum[5]), pack16<kB>(sum[6], sum[7]));
}

template <class T>
cudaError_t launch_sum(const ExpertArgs& a, const T* D, const float* wide, bool bf16, cudaStream_t stream) {
  const long long threads = (long long)a.T * (a.N / 8);
  const dim3 grid((unsigned)((threads + kThreads - 1) / kThreads));
  using Loaded = std::conditional_t<sizeof(T) == 2, Eight16, Eight32>;
  return bf16 ? launch_pdl(experts_sum_kernel<true, T, Loaded>, grid, dim3(kThreads), 0, stream, a, D, wide)
              : launch_pdl(experts_sum_kernel<false, T, Loaded>, grid, dim3(kThreads), 0, stream, a, D, wide);
}

// How a call is laid out.
struct Layout {
  int tile, parts, blocks;  // rows of an item, parts of K, column blocks
  int smem, per_sm;         // bytes of shared memory, blocks of an SM
};

// Dynamic shared memory: the warps' units of weights, the parts' rows (an octet
// is read whole, whatever of it there is).
int smem_bytes(int parts, int rows) {
  return kWarps * kWeightSlots * kSlotBytes + (kRowSlots * parts * rows + (rows + 7) / 8 * 8 - rows) * kRowBytes;
}

// Parts of K: of 1, 2 and 4 those with the fewest rounds of items (as many as
// are likely, were every choice as likely) times the work of an item, the
// fewer where two are alike: one token's gate and up over eight of 64 experts
// take 7.7 us in two parts, 11.1 in one. Items have 16 rows where there can be more
// than 8: with items of 8 gate and up of 32 tokens over 8 experts, top 2, take
// 115-120 us against 100-111, down of 100 over 64, top 8, 48 against 41, gate and up
// of 16 tokens over 64 the same 35-37. Nor has an item more rows than there are tokens, as many as an
// expert can have of the router: for a few tokens shared memory is small.
Layout choose_layout(const ExpertArgs& a, int sms) {
  const double experts = a.E * (1.0 - std::pow(1.0 - 1.0 / a.E, (double)choices(a)));
  Layout best = {};
  double least = 0;
  for (int parts = 1; parts <= 4; parts *= 2) {
    Layout l;
    const int rows = a.T <= 8 ? 8 : 16;
    l.tile = a.T < rows ? a.T : rows;
    l.parts = parts;
    const int per = kWarps / parts * kStripCols / (a.silu ? 2 : 1);  // results of an item
    l.blocks = ((a.silu ? a.N / 2 : a.N) + per - 1) / per;
    l.smem = smem_bytes(parts, l.tile);
    l.per_sm = 2 * (l.smem + 15 * 1024) <= 228 * 1024 ? 2 : 1;  // (beside it 14 KB of the kernel's own and 1 KB)
    const double tiles = experts + (double)choices(a) / rows / 2;
    const double cost = std::ceil(tiles * l.blocks / (sms * l.per_sm)) / parts;
    if (parts == 1 || cost < 0.95 * least) {
      least = cost;
      best = l;
    }
  }
  return best;
}

template <bool kB, int KS, bool kPairs>
cudaError_t launch_decode_kernel(DecodeParams p, const Layout& l, int sms, cudaStream_t stream) {
  const ExpertArgs& a = p.a;
  const auto kernel = experts_decode_kernel<kB, KS, kPairs>;
  cudaError_t e = set_max_smem_once(reinterpret_cast<const void*>(kernel),
                                    kWarps * kWeightSlots * kSlotBytes + kRowSlots * KS * kRows * kRowBytes);
  if (e != cudaSuccess) return e;
  p.blocks = l.blocks;
  p.tile = l.tile;
  // no more blocks than there are items of the router's choices
  const long long most = (long long)(choices(a) / (l.tile < 8 ? 8 : l.tile) + (choices(a) < a.E + 1 ? choices(a) : a.E + 1)) * l.blocks;
  const long long resident = (long long)l.per_sm * sms;
  const dim3 grid((unsigned)(most < resident ? most : resident));
  return launch_pdl(kernel, grid, dim3(kThreads), (size_t)l.smem, stream, p);
}

template <bool kB, int KS>
cudaError_t launch_decode_ks(const DecodeParams& p, const Layout& l, int sms, cudaStream_t stream) {
  return p.a.group == 2 * kAtomK ? launch_decode_kernel<kB, KS, true>(p, l, sms, stream)
                                 : launch_decode_kernel<kB, KS, false>(p, l, sms, stream);
}

template <bool kB>
cudaError_t launch_experts_decode_t(const DecodeParams& p, int sms, cudaStream_t stream) {
  const Layout l = choose_layout(p.a, sms);
  return l.parts == 4   ? launch_decode_ks<kB, 4>(p, l, sms, stream)
         : l.parts == 2 ? launch_decode_ks<kB, 2>(p, l, sms, stream)
                        : launch_decode_ks<kB, 1>(p, l, sms, stream);
}

}  // namespace

size_t experts_decode_workspace_bytes(int choices, int N, bool combine) {
  return combine ? kWorkspaceFlags + (size_t)choices * N * sizeof(float) : 0;
}

cudaError_t launch_experts_decode(ExpertArgs a, bool bf16, void* workspace, cudaStream_t stream) {
  cudaError_t e = device_error_word(&a.err);
  if (e != cudaSuccess) return e;
  DecodeParams p = {a, workspace ? reinterpret_cast<float*>(static_cast<uint8_t*>(workspace) + kWorkspaceFlags) : nullptr, 0, 0};
  const int sms = device_sms();
  e = bf16 ? launch_experts_decode_t<true>(p, sms, stream) : launch_experts_decode_t<false>(p, sms, stream);
  return e != cudaSuccess || !a.combine ? e : launch_sum(a, p.D, nullptr, bf16, stream);
}

cudaError_t launch_experts_sum(const ExpertArgs& a, const uint16_t* D, const float* wide, bool bf16, cudaStream_t stream) {
  return launch_sum(a, D, wide, bf16, stream);
}

}  // namespace w4a16
