// Attention of one new token per sequence over the paged cache, split over
// the cache's length and joined.
//
// For the query rows of one key/value head (the group of G = heads / kv_heads
// query heads that share it, at most 16 at a time) and the cached keys and
// values j < n:
//   s_j = scale q.k_j,  o = sum_j 2^(x_j - m) v_j / l,  x_j = s_j log2 e,
// with the running maximum m of x and the sum l of 2^(x_j - m). Two parts of
// the keys with (m1, l1, o1) and (m2, l2, o2), o unnormalised, join to
// m = max(m1, m2), l = sum l_i 2^(m_i - m), o = sum o_i 2^(m_i - m).
//
// Bound: HBM bytes, every cached key and value read once (2 n D values per
// key/value head; the queries and results are small). So the kernel is built
// around bytes in flight: each warp streams its own tiles (4 KiB of keys, 4
// KiB of values) through a private ring of kStages slots with 16-byte
// asynchronous copies, without any barrier between warps; two blocks of four
// warps per SM hold 128 KiB in flight. Both products run on mma.sync m16n8k16
// (the group's rows are its 16 rows): at 24 B per clock and SM they need a
// tenth of its rate, and a tcgen05 tile of 128 rows would be filled with at
// most 16.
//
// Work: all (sequence, head, step of four tiles) triples in one line, cut into
// equal runs, one per block, from the lengths on the device. A run may begin
// and end inside an item (sequence, head); such an item's parts go to the
// workspace as fp32 (m, l, o), and the last of its blocks to arrive joins
// them in the order of the parts, whichever block that is: results do not
// depend on the order of arrival. The ring runs on across items.
#include "common.cuh"
#include "kernels.h"
#include "layer.cuh"

namespace w4a16 {
namespace {

constexpr int kWarps = 4;
constexpr int kThreads = kWarps * 32;
constexpr int kStages = 3;
constexpr int kTileBytes = 4096;         // of keys, and as many of values
constexpr int kRows = 16;                // query rows of an item
constexpr int kJoinRows = 8;             // rows joined at a time
constexpr float kLog2e = 1.4426950408889634f, kLn2 = 0.6931471805599453f;

// Column of value d of row r in the joining rows: rows that are stored
// together fall on different banks (two rows of 16 floats at a time with k8,
// four of 8 without). No padding: two blocks' shared memory just fits an SM.
template <bool k8>
__device__ __forceinline__ int join_at(int r, int d) { return d ^ (k8 ? (r & 1) * 16 : (r & 3) * 8); }

template <int D>
struct Smem {
  uint8_t ring[kWarps][kStages][2][kTileBytes];
  float o[kWarps][kJoinRows][D];  // columns permuted by join_at
  float ml[2][kWarps][kRows];         // maxima, sums
  float top[kRows], sum[kRows];       // of the item
  int scan[kWarps];
  int start[3];  // sequence, steps before it, total
  int last;
};

struct DecodeArgs {
  AttnArgs a;
  int* arrived;     // one counter per block: parts of the split item that it begins
  float* parts;     // [blocks][2] of kPartFloats
  int group, tiles;  // query heads per key/value head, 16-row tiles of them
};

static_assert(sizeof(Smem<128>) <= (227 * 1024 + 1024) / 2 - 1024, "two blocks per SM");

template <int D>
constexpr int kPartFloats = kRows * (D + 2);

__device__ __forceinline__ void cp16(uint32_t dst, const void* src, bool valid) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(valid ? 16 : 0) : "memory");
}
__device__ __forceinline__ void cp_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void cp_wait() { asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory"); }

__device__ __forceinline__ void ldsm4(uint32_t (&r)[4], uint32_t addr) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0, %1, %2, %3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]) : "r"(addr) : "memory");
}
__device__ __forceinline__ void ldsm4t(uint32_t (&r)[4], uint32_t addr) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0, %1, %2, %3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]) : "r"(addr) : "memory");
}
template <bool kB>
__device__ __forceinline__ void mma(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  if (kB)
    asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
                 "{%0, %1, %2, %3};"
                 : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
                 : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
  else
    mma_16816(c, a[0], a[1], a[2], a[3], b0, b1);
}
__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

// Byte offset of 16-byte chunk c of row r in a tile of kRowBytes-byte rows:
// chunks are permuted so that the 8 rows of a matrix load fall on different
// banks.
template <int kRowBytes>
__device__ __forceinline__ uint32_t tile_at(int r, int c) {
  if (kRowBytes == 64) return (uint32_t)(((r >> 1) * 8 + (((r & 1) * 4 + c) ^ ((r >> 1) & 3))) * 16);
  return (uint32_t)(r * kRowBytes + ((c ^ (r & 7)) * 16));
}

// A place in the line of work: the steps [step, end) of an item, within the
// run's remaining `left` steps.
struct Place {
  int b, item;  // sequence; head * tiles + 16-row tile
  int step, steps, len;
};

template <int kStep>
__device__ __forceinline__ int steps_of(int len) {
  return len > 0 ? (len + kStep - 1) / kStep : 1;  // an empty item still writes its result
}

// kB: 16-bit values are bf16, else fp16; k8: e4m3 cache (its products in
// fp16, which holds every e4m3 code).
template <bool kB, bool k8, int D>
__global__ void __launch_bounds__(kThreads, 2) attn_decode_kernel(const DecodeArgs p) {
  constexpr int kRowBytes = D * (k8 ? 1 : 2);
  constexpr int kTok = kTileBytes / kRowBytes;  // tokens per tile
  constexpr int kStep = kWarps * kTok;
  constexpr int kChunks = kRowBytes / 16;
  constexpr int kPages = kTok / 16;  // most pages of a tile
  constexpr bool kP = kB && !k8;     // products in bf16
  constexpr int kSteps16 = D / 16;   // k-steps of the score product

  extern __shared__ __align__(128) uint8_t smem_raw[];
  Smem<D>& sm = *reinterpret_cast<Smem<D>*>(smem_raw);
  const AttnArgs& a = p.a;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, g = lane >> 2, t = lane & 3;
  const int items = a.cache.kv_heads * p.tiles;  // per sequence

  allow_dependent_launch();
  grid_dependency_wait();

  // the line's length, and where this block's run begins in it
  auto scan = [&](int v) {  // inclusive over the block; the total in `total`
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int u = __shfl_up_sync(0xffffffffu, v, o);
      if (lane >= o) v += u;
    }
    if (lane == 31) sm.scan[warp] = v;
    __syncthreads();
    int before = 0, all = 0;
#pragma unroll
    for (int w = 0; w < kWarps; ++w) {
      if (w < warp) before += sm.scan[w];
      all += sm.scan[w];
    }
    __syncthreads();
    return make_int2(v + before, all);
  };
  long long total = 0;
  for (int b0 = 0; b0 < a.batch; b0 += kThreads) {
    const int v = b0 + tid < a.batch ? steps_of<kStep>(seq_length(a, b0 + tid)) : 0;
    total += (long long)scan(v).y * items;
  }
  // at least a step per block, so that every block from an item's first to
  // its last has a part of it
  const long long blocks = min((long long)gridDim.x, total), me = blockIdx.x;
  if (me >= blocks) return;
  const long long begin = me * total / blocks, end = (me + 1) * total / blocks;
  long long carry = 0;
  for (int b0 = 0; b0 < a.batch; b0 += kThreads) {
    const int v = b0 + tid < a.batch ? steps_of<kStep>(seq_length(a, b0 + tid)) : 0;
    const int2 s = scan(v);
    const long long hi = carry + (long long)s.x * items, lo = hi - (long long)v * items;
    if (lo <= begin && begin < hi) {
      sm.start[0] = b0 + tid;
      sm.start[1] = (int)((begin - lo) / v);
      sm.start[2] = (int)((begin - lo) % v);
    }
    carry += (long long)s.y * items;
  }
  __syncthreads();

  Place load;  // what the ring loads next
  load.b = sm.start[0];
  load.item = sm.start[1];
  load.step = sm.start[2];
  load.len = seq_length(a, load.b);
  load.steps = steps_of<kStep>(load.len);
  Place cur = load;  // what the products take next
  long long load_left = end - begin, left = end - begin;
  auto advance = [&](Place& q) {  // by one step
    if (++q.step < q.steps) return;
    q.step = 0;
    if (++q.item < items) return;
    q.item = 0;
    if (++q.b < a.batch) {
      q.len = seq_length(a, q.b);
      q.steps = steps_of<kStep>(q.len);
    }
  };

  const uint32_t ring = (uint32_t)__cvta_generic_to_shared(&sm.ring[warp][0][0][0]);
  const int shift = a.cache.page_shift, mask = (1 << shift) - 1;
  auto issue = [&](int slot) {  // the next step's tile of this warp into a ring slot
    if (load_left > 0) {
      --load_left;
      const int tok0 = (load.step * kWarps + warp) * kTok;
      if (tok0 < load.len) {
        const int head = load.item / p.tiles;
        size_t page[kPages];
#pragma unroll
        for (int i = 0; i < kPages; ++i) {
          const int tok = tok0 + 16 * i;
          // a place of the page's rows of this head, in bytes
          page[i] = tok < load.len
                        ? ((((size_t)page_of(a, load.b, tok >> shift) * a.cache.kv_heads + head) << shift) + (tok & mask)) *
                              kRowBytes
                        : 0;
        }
        const uint32_t dst = ring + slot * (2 * kTileBytes);
        const uint8_t* k = static_cast<const uint8_t*>(a.cache.k);
        const uint8_t* v = static_cast<const uint8_t*>(a.cache.v);
#pragma unroll
        for (int i = 0; i < kTileBytes / 512; ++i) {
          const int u = i * 32 + lane, r = u / kChunks, c = u % kChunks;
          const bool valid = tok0 + r < load.len;
          const size_t at = valid ? page[(i * 32 / kChunks) / 16] + (size_t)(r & 15) * kRowBytes + c * 16 : 0;
          cp16(dst + tile_at<kRowBytes>(r, c), k + at, valid);
          cp16(dst + kTileBytes + tile_at<kRowBytes>(r, c), v + at, valid);
        }
      }
      advance(load);
    }
    cp_commit();
  };
#pragma unroll
  for (int i = 0; i < kStages - 1; ++i) issue(i);
  int slot = 0;

  while (left > 0) {
    // one item's steps of this run
    const int head = cur.item / p.tiles, row0 = (cur.item % p.tiles) * kRows;
    const int rows = min(kRows, p.group - row0);
    const bool starts = cur.step == 0;
    const int n = (int)min((long long)(cur.steps - cur.step), left);
    const bool ends = cur.step + n == cur.steps;

    // the queries as A fragments: rows g and g + 8; for the e4m3 cache in
    // fp16 with the dimensions of a k-step in the order its codes come in
    // (4t, 4t + 1 | 4t + 2, 4t + 3), each row divided by a power of two
    uint32_t qf[kSteps16][4];
    float mult[2];
#pragma unroll
    for (int half = 0; half < 2; ++half) {
      const int r = g + 8 * half;
      const uint16_t* q = a.q + (size_t)cur.b * a.ldq + (size_t)(head * p.group + row0 + (r < rows ? r : 0)) * D;
      float top = 0.f;
#pragma unroll
      for (int i = 0; i < kSteps16; ++i) {
#pragma unroll
        for (int w = 0; w < 2; ++w) {
          const int d = k8 ? 16 * i + 4 * t + 2 * w : 16 * i + 2 * t + 8 * w;
          const uint32_t v = r < rows ? *reinterpret_cast<const uint32_t*>(q + d) : 0;
          qf[i][half + 2 * w] = v;
          if (k8 && kB) {
            const float2 f = unpack16<true>(v);
            top = fmaxf(top, fmaxf(fabsf(f.x), fabsf(f.y)));
          }
        }
      }
      mult[half] = a.scale * kLog2e * (k8 ? a.cache.k_scale[head] : 1.f);
      if (k8 && kB) {
        top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 1));
        top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 2));
        const int e = top > 0.f ? ilogbf(top) : 0;  // |q| 2^-e < 2
#pragma unroll
        for (int i = 0; i < kSteps16; ++i)
#pragma unroll
          for (int w = 0; w < 2; ++w) {
            const float2 f = unpack16<true>(qf[i][half + 2 * w]);
            qf[i][half + 2 * w] = pack16<false>(scalbnf(f.x, -e), scalbnf(f.y, -e));
          }
        mult[half] = scalbnf(mult[half], e);
      }
    }

    float o[D / 8][4];
#pragma unroll
    for (int i = 0; i < D / 8; ++i)
#pragma unroll
      for (int j = 0; j < 4; ++j) o[i][j] = 0.f;
    float m[2] = {-INFINITY, -INFINITY}, l[2] = {0.f, 0.f};

    for (int k = 0; k < n; ++k) {
      cp_wait<kStages - 2>();
      __syncwarp();
      issue(slot == 0 ? kStages - 1 : slot - 1);  // into the slot read one step ago
      const int tok0 = (cur.step * kWarps + warp) * kTok;
      const uint32_t kt = ring + slot * (2 * kTileBytes), vt = kt + kTileBytes;
      if (tok0 < cur.len) {
        // scores: kTok tokens in blocks of 8
        float s[kTok / 8][4];
#pragma unroll
        for (int nb = 0; nb < kTok / 8; ++nb) {
          s[nb][0] = s[nb][1] = s[nb][2] = s[nb][3] = 0.f;
          const int r = nb * 8 + (lane & 7);
#pragma unroll
          for (int c = 0; c < kChunks; c += 4) {
            uint32_t b[4];
            ldsm4(b, kt + tile_at<kRowBytes>(r, c + (lane >> 3)));
            if (k8) {
#pragma unroll
              for (int i = 0; i < 4; ++i)
                mma<kP>(s[nb], qf[c + i], e4m3x2_to_half2(b[i] & 0xffffu), e4m3x2_to_half2(b[i] >> 16));
            } else {
              mma<kP>(s[nb], qf[c / 2], b[0], b[1]);
              mma<kP>(s[nb], qf[c / 2 + 1], b[2], b[3]);
            }
          }
        }
        float top[2] = {-INFINITY, -INFINITY};
#pragma unroll
        for (int nb = 0; nb < kTok / 8; ++nb)
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            const int tok = tok0 + nb * 8 + 2 * t + (j & 1);
            s[nb][j] = tok < cur.len ? s[nb][j] * mult[j >> 1] : -INFINITY;
            top[j >> 1] = fmaxf(top[j >> 1], s[nb][j]);
          }
        bool grew = false;
        float base[2];
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          top[h] = fmaxf(top[h], __shfl_xor_sync(0xffffffffu, top[h], 1));
          top[h] = fmaxf(top[h], __shfl_xor_sync(0xffffffffu, top[h], 2));
          grew |= top[h] > m[h];
          top[h] = fmaxf(m[h], top[h]);
          base[h] = top[h] == -INFINITY ? 0.f : top[h];
        }
        if (__any_sync(0xffffffffu, grew)) {
          float f[2];
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            f[h] = ex2(m[h] - base[h]);
            l[h] *= f[h];
            m[h] = top[h];
          }
#pragma unroll
          for (int i = 0; i < D / 8; ++i)
#pragma unroll
            for (int j = 0; j < 4; ++j) o[i][j] *= f[j >> 1];
        }
#pragma unroll
        for (int nb = 0; nb < kTok / 8; ++nb)
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            s[nb][j] = ex2(s[nb][j] - base[j >> 1]);
            l[j >> 1] += s[nb][j];
          }
        // values: 16 tokens per k-step, the probabilities rounded to 16 bits
        // for the product (relative 2^-11 or 2^-8 of each term)
#pragma unroll
        for (int ks = 0; ks < kTok / 16; ++ks) {
          uint32_t pa[4];
          pa[0] = pack16<kP>(s[2 * ks][0], s[2 * ks][1]);
          pa[1] = pack16<kP>(s[2 * ks][2], s[2 * ks][3]);
          pa[2] = pack16<kP>(s[2 * ks + 1][0], s[2 * ks + 1][1]);
          pa[3] = pack16<kP>(s[2 * ks + 1][2], s[2 * ks + 1][3]);
          const int r = ks * 16 + (lane & 15);
#pragma unroll
          for (int c = 0; c < kChunks; c += 2) {
            uint32_t b[4];
            ldsm4t(b, vt + tile_at<kRowBytes>(r, c + (lane >> 4)));
            if (k8) {
              // a register holds dimensions (2g, 2g + 1) of two tokens: the
              // even ones of both first, then the odd ones
#pragma unroll
              for (int i = 0; i < 2; ++i) {
                const uint32_t x = __byte_perm(b[2 * i], 0, 0x3120), y = __byte_perm(b[2 * i + 1], 0, 0x3120);
                mma<kP>(o[2 * (c + i)], pa, e4m3x2_to_half2(x & 0xffffu), e4m3x2_to_half2(y & 0xffffu));
                mma<kP>(o[2 * (c + i) + 1], pa, e4m3x2_to_half2(x >> 16), e4m3x2_to_half2(y >> 16));
              }
            } else {
              mma<kP>(o[c], pa, b[0], b[1]);
              mma<kP>(o[c + 1], pa, b[2], b[3]);
            }
          }
        }
      }
      slot = slot == kStages - 1 ? 0 : slot + 1;
      ++cur.step;
    }

    // join the warps
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      l[h] += __shfl_xor_sync(0xffffffffu, l[h], 1);
      l[h] += __shfl_xor_sync(0xffffffffu, l[h], 2);
      if (t == 0) {
        sm.ml[0][warp][g + 8 * h] = m[h];
        sm.ml[1][warp][g + 8 * h] = l[h];
      }
    }
    __syncthreads();
    if (tid < kRows) {
      float top = sm.ml[0][0][tid];
#pragma unroll
      for (int w = 1; w < kWarps; ++w) top = fmaxf(top, sm.ml[0][w][tid]);
      const float base = top == -INFINITY ? 0.f : top;
      float sum = 0.f;
#pragma unroll
      for (int w = 0; w < kWarps; ++w) sum += sm.ml[1][w][tid] * ex2(sm.ml[0][w][tid] - base);
      sm.top[tid] = top;
      sm.sum[tid] = sum;
    }
    const bool whole = starts && ends;
    float* part = p.parts + (size_t)(2 * me + (starts ? 1 : 0)) * kPartFloats<D>;
    const float v_scale = k8 ? a.cache.v_scale[head] : 1.f;
    const size_t out0 = (size_t)cur.b * a.heads + head * p.group + row0;
#pragma unroll
    for (int half = 0; half < 2; ++half) {
      if (half * kJoinRows >= rows) break;
      __syncthreads();  // the maxima are there, and the rows before these are read
      const float base = sm.top[g + 8 * half] == -INFINITY ? 0.f : sm.top[g + 8 * half];
      const float f = ex2(m[half] - base);
      float* row = &sm.o[warp][g][0];
      if (k8) {
        // (even, odd) pairs of blocks hold four dimensions in a row
#pragma unroll
        for (int i = 0; i < D / 8; i += 2)
          *reinterpret_cast<float4*>(row + join_at<k8>(g, 8 * i + 4 * t)) =
              make_float4(o[i][2 * half] * f, o[i + 1][2 * half] * f, o[i][2 * half + 1] * f, o[i + 1][2 * half + 1] * f);
      } else {
#pragma unroll
        for (int i = 0; i < D / 8; ++i)
          *reinterpret_cast<float2*>(row + join_at<k8>(g, 8 * i + 2 * t)) = make_float2(o[i][2 * half] * f, o[i][2 * half + 1] * f);
      }
      __syncthreads();
      const int some = min(kJoinRows, rows - half * kJoinRows);
      for (int u = tid; u < some * (D / 4); u += kThreads) {
        const int r = u / (D / 4), d = u % (D / 4) * 4, row = half * kJoinRows + r;
        float4 v = *reinterpret_cast<const float4*>(&sm.o[0][r][join_at<k8>(r, d)]);
#pragma unroll
        for (int w = 1; w < kWarps; ++w) {
          const float4 x = *reinterpret_cast<const float4*>(&sm.o[w][r][join_at<k8>(r, d)]);
          v.x += x.x, v.y += x.y, v.z += x.z, v.w += x.w;
        }
        if (whole) {
          const float l1 = sm.sum[row], inv = l1 > 0.f ? v_scale / l1 : 0.f;
          *reinterpret_cast<uint2*>(a.out + (out0 + row) * D + d) =
              make_uint2(pack16<kB>(v.x * inv, v.y * inv), pack16<kB>(v.z * inv, v.w * inv));
        } else {
          *reinterpret_cast<float4*>(part + row * D + d) = v;
        }
      }
    }
    if (tid < rows) {
      if (whole) {
        if (a.lse) a.lse[out0 + tid] = sm.sum[tid] > 0.f ? sm.top[tid] * kLn2 + logf(sm.sum[tid]) : -INFINITY;
      } else {
        part[kRows * D + tid] = sm.top[tid];
        part[kRows * D + kRows + tid] = sm.sum[tid];
      }
    }

    if (!whole) {
      // this item's steps in the line, and the blocks that have a part of it
      const long long at = begin + (end - begin - left) - (cur.step - n);  // the item's first step
      const long long first = ((at + 1) * blocks - 1) / total, final = ((at + cur.steps) * blocks - 1) / total;
      __threadfence();
      __syncthreads();
      if (tid == 0) sm.last = atomicAdd(p.arrived + first, 1) == (int)(final - first);
      __syncthreads();
      if (sm.last) {
        __threadfence();
        const int count = (int)(final - first) + 1;
        auto part_of = [&](int i) { return p.parts + (size_t)(2 * (first + i) + (i == 0 ? 1 : 0)) * kPartFloats<D>; };
        // maxima and sums: 8 threads per row over the parts
        {
          const int r = tid >> 3, j = tid & 7;
          float top = -INFINITY, sum = 0.f;
          if (r < rows)
            for (int i = j; i < count; i += 8) top = fmaxf(top, __ldcg(part_of(i) + kRows * D + r));
#pragma unroll
          for (int w = 1; w < 8; w <<= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, w));
          const float base = top == -INFINITY ? 0.f : top;
          if (r < rows)
            for (int i = j; i < count; i += 8)
              sum += __ldcg(part_of(i) + kRows * D + kRows + r) * ex2(__ldcg(part_of(i) + kRows * D + r) - base);
#pragma unroll
          for (int w = 1; w < 8; w <<= 1) sum += __shfl_xor_sync(0xffffffffu, sum, w);
          if (j == 0) {
            sm.top[r] = top;
            sm.sum[r] = sum;
          }
        }
        __syncthreads();
        for (int u = tid; u < rows * (D / 4); u += kThreads) {
          const int r = u / (D / 4), d = u % (D / 4) * 4;
          const float base = sm.top[r] == -INFINITY ? 0.f : sm.top[r];
          float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 8
          for (int i = 0; i < count; ++i) {
            const float* q = part_of(i);
            const float f = ex2(__ldcg(q + kRows * D + r) - base);
            const float4 x = __ldcg(reinterpret_cast<const float4*>(q + r * D + d));
            v.x = fmaf(x.x, f, v.x), v.y = fmaf(x.y, f, v.y), v.z = fmaf(x.z, f, v.z), v.w = fmaf(x.w, f, v.w);
          }
          const float l1 = sm.sum[r], inv = l1 > 0.f ? v_scale / l1 : 0.f;
          *reinterpret_cast<uint2*>(a.out + (out0 + r) * D + d) =
              make_uint2(pack16<kB>(v.x * inv, v.y * inv), pack16<kB>(v.z * inv, v.w * inv));
        }
        if (a.lse && tid < rows)
          a.lse[out0 + tid] = sm.sum[tid] > 0.f ? sm.top[tid] * kLn2 + logf(sm.sum[tid]) : -INFINITY;
        if (tid == 0) p.arrived[first] = 0;  // left zero for the next call
      }
    }
    left -= n;
    // to the next item
    cur.step = 0;
    if (++cur.item == items) {
      cur.item = 0;
      if (++cur.b < a.batch) {
        cur.len = seq_length(a, cur.b);
        cur.steps = steps_of<kStep>(cur.len);
      }
    }
    __syncthreads();  // the shared maxima and rows are free again
  }
  cp_wait<0>();
}

template <bool kB, bool k8, int D>
cudaError_t launch(const DecodeArgs& p, int blocks, cudaStream_t stream) {
  auto kern = attn_decode_kernel<kB, k8, D>;
  cudaError_t e = set_max_smem_once(reinterpret_cast<const void*>(kern), (int)sizeof(Smem<D>));
  if (e != cudaSuccess) return e;
  return launch_pdl(kern, dim3((unsigned)blocks), dim3(kThreads), sizeof(Smem<D>), stream, p);
}

constexpr size_t kFlagBytes = 32768;

}  // namespace

size_t attn_decode_workspace_bytes(int head_dim, int sms) {
  return kFlagBytes + (size_t)(2 * sms) * 2 * kRows * (head_dim + 2) * sizeof(float);
}

cudaError_t launch_attn_decode(const AttnArgs& args, int head_dim, bool bf16, bool e4m3, void* workspace, int sms,
                               cudaStream_t stream) {
  if (args.batch == 0) return cudaSuccess;
  DecodeArgs p;
  p.a = args;
  cudaError_t e = device_error_word(&p.a.err);
  if (e != cudaSuccess) return e;
  p.arrived = static_cast<int*>(workspace);
  p.parts = reinterpret_cast<float*>(static_cast<uint8_t*>(workspace) + kFlagBytes);
  p.group = args.heads / args.cache.kv_heads;
  p.tiles = (p.group + kRows - 1) / kRows;
  const int blocks = 2 * sms;
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
