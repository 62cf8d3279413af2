// W4A16 products grouped by expert, for few rows per expert, and the weighted
// sum over a token's experts.
//
// Choice f of expert e: Y[f][n] = sum_k A[f or f / top][k] (q - z) s [e][k][n],
// with the gate/up epilogue silu(gate) * up of columns [gate | up], or summed
// over a token's choices with their weights.
//
// Every expert that has rows streams its packed weights once per 16 rows, so
// the bound is HBM bytes, and for a token or two the chain offsets - rows -
// activations and weights - sums. A block takes up to 16 rows of one expert
// and 128 / KS columns; its 8 warps take a strip of 16 columns each and one of
// KS parts of K, so that few rows still spread over all SMs. A lane loads its
// four words of an atom with 16 bytes, eight atoms ahead; the activations come
// to shared memory by asynchronous copies, gathered by row. The codes enter
// mma.sync m16n8k16 as exact 16-bit numbers without a multiplication: fp16
// takes q masked in place as the subnormal q 2^-24 (the odd pairs one nibble
// higher, summed apart and divided by 16), bf16 takes 128 + q put together by
// byte permutes; the zero point, in the same form, is subtracted exactly. Each
// group's fp32 sum is multiplied by its scale. So the weights are (q - z) s
// unrounded, the sums fp32, and the result is rounded once.
//
// Combined, each choice's product goes to the workspace in fp32, and a second
// kernel adds a token's rows, multiplied by their weights, in the order of its
// choices: no atomics, the same result every time.
#include <cuda_bf16.h>

#include "experts.cuh"

namespace w4a16 {
namespace {

constexpr int kThreads = 256;
constexpr int kWarps = 8;
constexpr int kRows = 16;      // rows of a block
constexpr int kUnit = 8;       // atoms loaded ahead
constexpr int kRowPad = 64;    // bytes: neighbouring rows in opposite halves of the banks
constexpr uint32_t kFull = 0xffffffffu;

struct DecodeParams {
  ExpertArgs a;
  float* D;      // combined: [choices][N]
  int chunk;     // atoms of a part in one piece of the activations
  int pieces;    // pieces of a part
};

__device__ __forceinline__ void copy16(uint32_t to, const void* from) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(to), "l"(from) : "memory");
}
__device__ __forceinline__ void copies_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void copies_wait() { asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory"); }

template <bool kB>
__device__ __forceinline__ void mma(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                    uint32_t b1) {
  if (kB)
    asm("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
        "{%0, %1, %2, %3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
  else
    asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
        "{%0, %1, %2, %3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// A zero point in the codes' form: lo for pairs 0 and 1, hi for 2 and 3 (bf16:
// one form for all).
template <bool kB>
struct Zero {
  uint32_t lo, hi;
  __device__ __forceinline__ explicit Zero(uint32_t z) {
    if (kB) {
      lo = hi = 0x43004300u | z | (z << 16);
    } else {
      lo = z | (z << 16);
      hi = lo << 4;
    }
  }
};

// The four pairs of a word minus the zero point: (k 0, 1), (2, 3), (4, 5),
// (6, 7); exact. fp16: (q - z) 2^-24 in the first two, 16 times that in the
// others; bf16: q - z.
template <bool kB>
__device__ __forceinline__ void codes(uint32_t w, const Zero<kB>& z, uint32_t (&c)[4]) {
  if (kB) {
    const uint32_t t = w & 0x0F0F0F0Fu, u = (w >> 4) & 0x0F0F0F0Fu;
    c[0] = __byte_perm(t, 0x43434343u, 0x4240);
    c[1] = __byte_perm(t, 0x43434343u, 0x4341);
    c[2] = __byte_perm(u, 0x43434343u, 0x4240);
    c[3] = __byte_perm(u, 0x43434343u, 0x4341);
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

// The row tile `y` of the launch: expert, first row and rows (0: none). The
// experts' tiles of kRows rows follow one another, those of no expert (e = E)
// last. By a whole warp.
struct RowTile {
  int e, first, n;
};
__device__ __forceinline__ RowTile find_tile(const ExpertArgs& a, int y, int lane) {
  int sum = 0;
  for (int e0 = 0; e0 <= a.E; e0 += 32) {
    const int e = e0 + lane;
    int begin = 0, end = 0;
    if (e <= a.E) {
      begin = offset_of(a, e);
      end = e < a.E ? offset_of(a, e + 1) : choices(a);
    }
    const int tiles = end > begin ? (end - begin + kRows - 1) / kRows : 0;
    int s = tiles;
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
      const int u = __shfl_up_sync(kFull, s, d);
      if (lane >= d) s += u;
    }
    s += sum;
    const uint32_t past = __ballot_sync(kFull, s > y);
    if (past) {
      const int l = __ffs(past) - 1;
      const int at = y - __shfl_sync(kFull, s - tiles, l);
      const int first = __shfl_sync(kFull, begin, l) + at * kRows, last = __shfl_sync(kFull, end, l);
      return {e0 + l, first, min(kRows, last - first)};
    }
    sum = __shfl_sync(kFull, s, 31);
  }
  return {0, 0, 0};
}

// One unit of a warp's strip: words, and the groups' scales and zero points:
// lane 8 i + c holds those of columns c and c + 8 of groups i and i + 4 from
// the unit's first group on.
struct Unit {
  uint4 w[kUnit];
  uint32_t s[2], z[2];
};

template <bool kB, int KS>
struct Strip {
  const DecodeParams& p;
  int strip;      // of all experts' columns; -1: none
  int end;        // one past the part's last atom
  int natoms, apg, G, lane;

  __device__ __forceinline__ void load(Unit& u, int a0, int n) const {
    const ExpertArgs& a = p.a;
    const uint4* base = reinterpret_cast<const uint4*>(a.Wq);
    const uint4* w = base + ((size_t)strip * natoms + a0) * 32 + lane;
    const size_t all = (size_t)a.E * a.N * a.K / 32;
#pragma unroll
    for (int j = 0; j < kUnit; ++j)
      if (j < n) u.w[j] = ldg_stream(ld_at(w + 32 * j, base, all, a.err));
    const int g0 = a0 / apg, g1 = (a0 + n - 1) / apg;
    const uint32_t* sp = reinterpret_cast<const uint32_t*>(a.Sp);
    const uint8_t* zp = reinterpret_cast<const uint8_t*>(a.Zp);
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const int g = g0 + lane / 8 + 4 * i;
      if (g > g1) continue;
      const size_t at = ((size_t)strip * G + g) * 8 + lane % 8, n2 = (size_t)a.E * a.N * G / 2;
      u.s[i] = __ldg(ld_at(sp + at, sp, n2, a.err));
      u.z[i] = __ldg(ld_at(zp + at, zp, n2, a.err));
    }
  }

  // out += the unit's products with the rows in shared memory (`act`: the
  // lane's place in its first row at the unit's first atom).
  template <int MT>
  __device__ __forceinline__ void multiply(float (&out)[MT][4], const Unit& u, uint32_t act, uint32_t row_bytes, int a0,
                                           int n) const {
    const int g0 = a0 / apg;
    float lo[MT][4] = {}, hi[MT][4] = {};
    uint32_t zs = 0, zz = 0;
    int left = 0, g = 0;  // atoms left of the group, group of the unit
    left = apg - (a0 - g0 * apg);
    auto group = [&]() {
      const uint32_t s0 = g < 4 ? u.s[0] : u.s[1], z0 = g < 4 ? u.z[0] : u.z[1];
      zs = __shfl_sync(kFull, s0, (g & 3) * 8 + lane / 4);
      zz = __shfl_sync(kFull, z0, (g & 3) * 8 + lane / 4);
    };
    group();
#pragma unroll
    for (int j = 0; j < kUnit; ++j) {
      if (j >= n) break;
      const Zero<kB> z0(zz & 15u), z1((zz >> 4) & 15u);
      const uint32_t w[4] = {u.w[j].x, u.w[j].y, u.w[j].z, u.w[j].w};
#pragma unroll
      for (int s = 0; s < 2; ++s) {
        uint32_t c0[4], c1[4];
        codes<kB>(w[2 * s], z0, c0);
        codes<kB>(w[2 * s + 1], z1, c1);
#pragma unroll
        for (int m = 0; m < MT; ++m) {
          const uint4 b = tc::lds128(act + m * 8 * row_bytes + j * 128 + s * 64);
          mma<kB>(lo[m], c0[0], c1[0], c0[1], c1[1], b.x, b.y);
          mma<kB>(kB ? lo[m] : hi[m], c0[2], c1[2], c0[3], c1[3], b.z, b.w);
        }
      }
      if (--left == 0 || j + 1 == n) {
        const float scale = kB ? 1.f : 16777216.f;
        const float s0 = value16<false>(zs & 0xffffu) * scale, s1 = value16<false>(zs >> 16) * scale;
#pragma unroll
        for (int m = 0; m < MT; ++m)
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const float v = kB ? lo[m][i] : fmaf(hi[m][i], 0.0625f, lo[m][i]);
            out[m][i] = fmaf(v, i < 2 ? s0 : s1, out[m][i]);
            lo[m][i] = hi[m][i] = 0.f;
          }
        if (left == 0 && j + 1 < n) {
          left = apg;
          ++g;
          group();
        }
      }
    }
  }
};

// The piece `c` of every part's activations: rows of `chunk` atoms, parts
// after one another. All threads of the block.
template <int KS>
__device__ __forceinline__ void copy_piece(const DecodeParams& p, const int* src, int n, uint32_t to, int c, int natoms,
                                           int row_bytes, uint32_t dyn) {
  const int vecs = p.chunk * 8;  // of a row of a part
  for (int i = threadIdx.x; i < n * KS * vecs; i += kThreads) {
    const int v = i % vecs, r = i / vecs % n, part = i / vecs / n;
    const int begin = natoms * part / KS + c * p.chunk, end = natoms * (part + 1) / KS;
    if (begin + v / 8 >= end) continue;
    const uint16_t* from = p.a.A + (size_t)src[r] * p.a.K + begin * kAtomK + v * 8;
    const uint32_t at = to + (uint32_t)((part * kRows + r) * row_bytes + v * 16);
    if (in_smem(at, 16, dyn, p.a.err)) copy16(at, ld_at(from, p.a.A, a_elements(p.a) - 7, p.a.err));
  }
}

template <bool kB, int KS, int MT>
__device__ __forceinline__ void run_strip(const DecodeParams& p, const Strip<kB, KS>& st, const int* src, int n, int part,
                                          uint32_t buffers, int row_bytes, uint32_t dyn, float (&out)[2][4]) {
  const int lane = threadIdx.x % 32;
  const int begin = st.natoms * part / KS;
  const uint32_t piece_bytes = (uint32_t)(KS * kRows * row_bytes);
  const bool live = st.strip >= 0;
  Unit cur, next;
  float acc[MT][4] = {};
  // (weights first: they are what the block waits for)
  if (live && begin < st.end) st.load(cur, begin, min(kUnit, min(p.chunk, st.end - begin)));
  copy_piece<KS>(p, src, n, buffers, 0, st.natoms, row_bytes, dyn);
  copies_commit();
  for (int c = 0; c < p.pieces; ++c) {
    if (c + 1 < p.pieces) {
      copy_piece<KS>(p, src, n, buffers + ((c + 1) & 1) * piece_bytes, c + 1, st.natoms, row_bytes, dyn);
      copies_commit();
      copies_wait<1>();
    } else {
      copies_wait<0>();
    }
    __syncthreads();
    const uint32_t act = buffers + (c & 1) * piece_bytes + (uint32_t)((part * kRows + lane / 4) * row_bytes + (lane % 4) * 16);
    const int a1 = begin + c * p.chunk, a2 = min(a1 + p.chunk, st.end);
    if (live)
      for (int a0 = a1; a0 < a2; a0 += kUnit) {
        const int len = min(kUnit, a2 - a0), after = a0 + len;
        // the next unit, in this piece or the next
        if (after < st.end)
          st.load(next, after, after < a2 ? min(kUnit, a2 - after) : min(kUnit, min(p.chunk, st.end - after)));
        const uint32_t at = act + (uint32_t)(a0 - a1) * 128;
        if (in_smem(at, (uint32_t)((MT - 1) * 8 * row_bytes + (len - 1) * 128 + 80), dyn, p.a.err))
          st.template multiply<MT>(acc, cur, at, (uint32_t)row_bytes, a0, len);
        cur = next;
      }
    __syncthreads();  // the buffer is free for the piece after the next
  }
#pragma unroll
  for (int m = 0; m < 2; ++m)
#pragma unroll
    for (int i = 0; i < 4; ++i) out[m][i] = m < MT ? acc[m < MT ? m : 0][i] : 0.f;
}

template <bool kB, int KS>
__global__ void __launch_bounds__(kThreads, 2) experts_decode_kernel(const DecodeParams p) {
  constexpr int S = kWarps / KS;        // strips of a block
  constexpr int kCols = S * kStripCols;
  constexpr int kRed = kCols + 4;       // floats of a row of partial sums
  extern __shared__ __align__(16) uint8_t dynamic[];
  __shared__ float red[KS][kRows][kRed];
  __shared__ int src[kRows], of[kRows];
  __shared__ RowTile tile;
  const ExpertArgs& a = p.a;
  const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
  const uint32_t dyn = (uint32_t)__cvta_generic_to_shared(dynamic);
  allow_dependent_launch();
  grid_dependency_wait();
  if (warp == 0) {
    const RowTile t = find_tile(a, blockIdx.x, lane);
    if (lane == 0) tile = t;
    if (lane < kRows) {
      const int f = lane < t.n ? choice_of(a, t.first + lane) : -1;
      of[lane] = f;
      src[lane] = f < 0 ? 0 : a.per_choice ? f : f / a.top;
    }
  }
  __syncthreads();
  const RowTile t = tile;
  if (t.n <= 0) return;
  const int half = a.N / 2, width = a.silu ? half : a.N;       // of a result's row
  const int cols = a.silu ? kCols / 2 : kCols;                 // of this block
  const int n0 = blockIdx.y * cols;
  if (t.e == a.E) {  // choices of no expert
    if (!a.combine)
      for (int i = threadIdx.x; i < t.n * cols; i += kThreads) {
        const int r = i / cols, n = n0 + i % cols;
        uint16_t* y = a.Y + (size_t)of[r] * width + n;
        if (of[r] >= 0 && n < width && in_buf(y, a.Y, (size_t)choices(a) * width, a.err)) *y = 0;
      }
    return;
  }
  // this warp's strip: with silu the block's first half are gate columns, the
  // second the up columns of the same results
  const int part = warp / S, w = warp % S;
  int strip = blockIdx.y * S + w;
  bool live = strip < a.N / kStripCols;
  if (a.silu) {
    const int i = blockIdx.y * (S / 2) + w % (S / 2);
    live = i < half / kStripCols;
    strip = i + (w < S / 2 ? 0 : half / kStripCols);
  }
  const int natoms = a.K / kAtomK;
  const Strip<kB, KS> st = {p, live ? t.e * (a.N / kStripCols) + strip : -1, natoms * (part + 1) / KS, natoms,
                            a.group / kAtomK, a.K / a.group, lane};
  const int row_bytes = p.chunk * 128 + kRowPad;
  float out[2][4];
  if (t.n <= 8)
    run_strip<kB, KS, 1>(p, st, src, t.n, part, dyn, row_bytes, dyn, out);
  else
    run_strip<kB, KS, 2>(p, st, src, t.n, part, dyn, row_bytes, dyn, out);
  // sums by token: lane (g, t) holds columns g, g + 8 of tokens 2t, 2t + 1
#pragma unroll
  for (int m = 0; m < 2; ++m)
#pragma unroll
    for (int i = 0; i < 4; ++i)
      red[part][m * 8 + (lane % 4) * 2 + (i & 1)][w * kStripCols + lane / 4 + (i & 2) * 4] = out[m][i];
  __syncthreads();
  for (int i = threadIdx.x; i < t.n * (cols / 2); i += kThreads) {
    const int r = i / (cols / 2), c = i % (cols / 2) * 2, n = n0 + c;
    if (of[r] < 0 || n >= width) continue;
    float v[2] = {0.f, 0.f}, u[2] = {0.f, 0.f};
#pragma unroll
    for (int k = 0; k < KS; ++k)
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        v[j] += red[k][r][c + j];
        if (a.silu) u[j] += red[k][r][kCols / 2 + c + j];
      }
    const size_t at = (size_t)of[r] * width + n, all = (size_t)choices(a) * width - 1;
    if (a.combine) {
      float* d = p.D + at;
      if (in_buf(d, p.D, all, a.err)) *reinterpret_cast<float2*>(d) = make_float2(v[0], v[1]);
    } else {
      if (a.silu) v[0] = silu_times(v[0], u[0]), v[1] = silu_times(v[1], u[1]);
      uint16_t* y = a.Y + at;
      if (in_buf(y, a.Y, all, a.err)) *reinterpret_cast<uint32_t*>(y) = pack16<kB>(v[0], v[1]);
    }
  }
}

// Eight columns of a row of products, 16-bit or fp32.
template <bool kB>
__device__ __forceinline__ void eight(const uint16_t* p, float (&v)[8]) {
  const uint4 u = __ldcs(reinterpret_cast<const uint4*>(p));
  const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float2 f = unpack16<kB>(w[i]);
    v[2 * i] = f.x, v[2 * i + 1] = f.y;
  }
}
template <bool kB>
__device__ __forceinline__ void eight(const float* p, float (&v)[8]) {
  const float4 a = __ldcs(reinterpret_cast<const float4*>(p)), b = __ldcs(reinterpret_cast<const float4*>(p) + 1);
  v[0] = a.x, v[1] = a.y, v[2] = a.z, v[3] = a.w, v[4] = b.x, v[5] = b.y, v[6] = b.z, v[7] = b.w;
}

// Y[t] = the weighted sum of the rows of D of token t's choices that have an
// expert, in their order, in fp32. One thread per eight columns.
template <bool kB, class T>
__global__ void __launch_bounds__(kThreads) experts_sum_kernel(const ExpertArgs a, const T* D) {
  allow_dependent_launch();
  grid_dependency_wait();
  const int vecs = a.N / 8;
  const long long i = (long long)blockIdx.x * kThreads + threadIdx.x;
  if (i >= (long long)a.T * vecs) return;
  const int t = (int)(i / vecs), n = (int)(i % vecs) * 8;
  float sum[8] = {};
#pragma unroll 4
  for (int j = 0; j < a.top; ++j) {
    const size_t f = (size_t)t * a.top + j;
    if (*ld_at(a.experts + f, a.experts, (size_t)choices(a), a.err) < 0) continue;
    const float w = *ld_at(a.weights + f, a.weights, (size_t)choices(a), a.err);
    float v[8];
    eight<kB>(ld_at(D + f * a.N + n, D, (size_t)choices(a) * a.N - 7, a.err), v);
#pragma unroll
    for (int k = 0; k < 8; ++k) sum[k] = fmaf(w, v[k], sum[k]);
  }
  uint16_t* y = a.Y + (size_t)t * a.N + n;
  if (in_buf(y, a.Y, (size_t)a.T * a.N - 7, a.err))
    *reinterpret_cast<uint4*>(y) = make_uint4(pack16<kB>(sum[0], sum[1]), pack16<kB>(sum[2], sum[3]),
                                              pack16<kB>(sum[4], sum[5]), pack16<kB>(sum[6], sum[7]));
}

template <class T>
cudaError_t launch_sum(const ExpertArgs& a, const T* D, bool bf16, cudaStream_t stream) {
  const long long threads = (long long)a.T * (a.N / 8);
  const dim3 grid((unsigned)((threads + kThreads - 1) / kThreads));
  return bf16 ? launch_pdl(experts_sum_kernel<true, T>, grid, dim3(kThreads), 0, stream, a, D)
              : launch_pdl(experts_sum_kernel<false, T>, grid, dim3(kThreads), 0, stream, a, D);
}

template <bool kB, int KS>
cudaError_t launch_decode_ks(DecodeParams p, cudaStream_t stream) {
  constexpr int S = kWarps / KS;
  const ExpertArgs& a = p.a;
  const int natoms = a.K / kAtomK, longest = (natoms + KS - 1) / KS;
  // the activations of all of K at once where they fit, else in pieces
  const auto bytes = [](int atoms) { return KS * kRows * (atoms * 128 + kRowPad); };
  p.chunk = bytes(longest) <= 72 * 1024 ? longest : KS == 1 ? 16 : 8;
  p.pieces = (longest + p.chunk - 1) / p.chunk;
  const int smem = bytes(p.chunk) * (p.pieces > 1 ? 2 : 1);
  cudaError_t e = set_max_smem_once(reinterpret_cast<const void*>(experts_decode_kernel<kB, KS>), 160 * 1024);
  if (e != cudaSuccess) return e;
  const int strips = a.N / kStripCols, per = a.silu ? S / 2 : S, n = a.silu ? strips / 2 : strips;
  const int tiles = choices(a) / kRows + (choices(a) < a.E + 1 ? choices(a) : a.E + 1);
  // (row tiles first: those of one expert read the same weights)
  const dim3 grid((unsigned)tiles, (unsigned)((n + per - 1) / per));
  return launch_pdl(experts_decode_kernel<kB, KS>, grid, dim3(kThreads), (size_t)smem, stream, p);
}

template <bool kB>
cudaError_t launch_experts_decode_t(const DecodeParams& p, int parts, cudaStream_t stream) {
  return parts == 4   ? launch_decode_ks<kB, 4>(p, stream)
         : parts == 2 ? launch_decode_ks<kB, 2>(p, stream)
                      : launch_decode_ks<kB, 1>(p, stream);
}

}  // namespace

size_t experts_decode_workspace_bytes(int choices, int N, bool combine) {
  return combine ? kWorkspaceFlags + (size_t)choices * N * sizeof(float) : 0;
}

cudaError_t launch_experts_decode(ExpertArgs a, bool bf16, void* workspace, cudaStream_t stream) {
  cudaError_t e = device_error_word(&a.err);
  if (e != cudaSuccess) return e;
  DecodeParams p = {a, workspace ? reinterpret_cast<float*>(static_cast<uint8_t*>(workspace) + kWorkspaceFlags) : nullptr, 0, 0};
  const int parts = 1;
  e = bf16 ? launch_experts_decode_t<true>(p, parts, stream) : launch_experts_decode_t<false>(p, parts, stream);
  return e != cudaSuccess || !a.combine ? e : launch_sum(a, p.D, bf16, stream);
}

cudaError_t launch_experts_sum(const ExpertArgs& a, const uint16_t* D, bool bf16, cudaStream_t stream) {
  return launch_sum(a, D, bf16, stream);
}

}  // namespace w4a16
