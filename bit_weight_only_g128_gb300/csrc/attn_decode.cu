// Attention of one new token per sequence over the paged cache, split over
// the cache's length and joined.
//
// For the query rows of one key/value head (the group of G = heads / kv_heads
// query heads that share it, 8 or 16 at a time) and the cached keys and
// values j < n:
//   s_j = scale q.k_j,  o = sum_j 2^(x_j - m) v_j / l,  x_j = s_j log2 e,
// with the running maximum m of x and the sum l of 2^(x_j - m). Two parts of
// the keys with (m1, l1, o1) and (m2, l2, o2), o unnormalised, join to
// m = max(m1, m2), l = sum l_i 2^(m_i - m), o = sum o_i 2^(m_i - m).
//
// Bound: HBM bytes, every cached key and value read once (2 n D values per
// key/value head; the queries and results are small). So the kernel is built
// around bytes in flight: each warp streams its own tiles (4 KiB of keys, 4
// KiB of values) through a private ring with 16-byte asynchronous copies,
// without any barrier between warps. Both products run on mma.sync m16n8k16
// with the tokens (keys) and the dimensions (values) as its 16 rows and the
// group's heads as its 8 columns:
//   S^T = K Q^T (16 tokens x 8 heads),  O^T += V^T P^T (16 dims x 8 heads),
// P^T being S^T's accumulators through one 8 x 8 transpose per 8 tokens. At 24
// B per clock and SM they need a twentieth of its rate; a tcgen05 tile of 128
// rows would be filled with at most 16.
//
// Measured, back to back: 64 x 8190 tokens, 64 heads over 8, fp16: 306 to 312
// us, 6870 to 7030 GB/s; 16 x up to 4096, 32 heads, bf16: 85 us, 6380 GB/s; 3 x
// 100003, 64 heads over 8, e4m3: 95 us, 6440 GB/s; 1 x 777: 8.2 us on the
// device, 8.8 a call. More than 16 heads per key/value head read the cache once
// per 16 of them: 16 x 8192, 64 heads over 1: 41 us for 67 MB.
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
constexpr int kTileBytes = 4096;  // of keys, and as many of values
constexpr size_t kFlagBytes = 32768;  // of the workspace: arrival counters, zero between calls
constexpr float kLog2e = 1.4426950408889634f, kLn2 = 0.6931471805599453f;

// Blocks per SM and ring slots of a warp by the heads of an item: 8 heads'
// accumulators leave registers for three blocks, whose warps cover each
// other's item changes; the rings fill what shared memory is left. (64 x 8190,
// 64 heads over 8: 310 us, 6930 GB/s, with a slot filled at the top of the step
// after it was read; 318 us with every slot filled as soon as it is read.)
template <int kHeads>
constexpr int kBlocks = kHeads == 8 ? 3 : 2;
template <int kHeads>
constexpr int kStages = kHeads == 8 ? 2 : 3;
constexpr int kJoinHeads = 4;  // heads joined at a time

// Column of dimension d of head h in the joining rows: heads that are stored
// together fall on different banks.
__device__ __forceinline__ int join_at(int h, int d) { return d ^ (((h >> 1) & 3) * 8); }

template <int D, int kHeads>
struct Smem {
  uint8_t ring[kWarps][kStages<kHeads>][2][kTileBytes];
  float o[kWarps][kJoinHeads][D];
  float ml[2][kWarps][kHeads];  // maxima, sums
  float top[kHeads], sum[kHeads];  // of the item
  int scan[kWarps];
  int start[4];  // sequence, item and step where the run begins, the sequence's length
  int last;
};
static_assert(sizeof(Smem<128, 8>) + 1024 <= 228 * 1024 / kBlocks<8>, "blocks per SM");
static_assert(sizeof(Smem<128, 16>) + 1024 <= 228 * 1024 / kBlocks<16>, "blocks per SM");

struct DecodeArgs {
  AttnArgs a;
  int* arrived;  // one counter per block: parts of the split item that it begins
  float* parts;  // [blocks][2] of kPartFloats
  size_t part_floats;  // of all of them
  int group, tiles;  // query heads per key/value head, items of kHeads of them
  float mult;        // |scale| log2 e
  uint32_t negate;   // sign bits of a pair of queries, where scale < 0
};

template <int D, int kHeads>
constexpr int kPartFloats = kHeads * (D + 2);

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
// An 8 x 8 matrix of 16-bit values, two of a row per lane, transposed.
__device__ __forceinline__ uint32_t transpose8(uint32_t v) {
  uint32_t r;
  asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(r) : "r"(v));
  return r;
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
template <bool kB, bool k8, int D, int kHeads>
__global__ void __launch_bounds__(kThreads, kBlocks<kHeads>) attn_decode_kernel(const DecodeArgs p) {
  constexpr int kRowBytes = D * (k8 ? 1 : 2);
  constexpr int kTok = kTileBytes / kRowBytes;  // tokens per tile
  constexpr int kStep = kWarps * kTok;
  constexpr int kChunks = kRowBytes / 16;
  constexpr int kPages = kTok / 16;   // most pages of a tile
  constexpr bool kP = kB && !k8;      // products in bf16
  constexpr int kNb = kHeads / 8;     // column blocks of heads
  constexpr int kSlots = kStages<kHeads>;

  extern __shared__ __align__(128) uint8_t smem_raw[];
  Smem<D, kHeads>& sm = *reinterpret_cast<Smem<D, kHeads>*>(smem_raw);
  const AttnArgs& a = p.a;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, g = lane >> 2, t = lane & 3;
  const int items = a.cache.kv_heads * p.tiles;  // per sequence

  allow_dependent_launch();
  grid_dependency_wait();

  // the line's length, and where this block's run begins in it
  auto scan = [&](int v) {  // inclusive over the block, and the total
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
  int own_len = 0;  // of the sequence of steps_at
  auto steps_at = [&](int b) {
    if (b >= a.batch) return 0;
    own_len = seq_length(a, b);
    return steps_of<kStep>(own_len);
  };
  const long long me = blockIdx.x;
  long long total = 0, blocks = 0, begin = 0, end = 0;
  // a * b / c, in 32 bits where the line is short (a 64-bit division takes
  // longer than the load of the lengths)
  auto share = [&](long long a1, long long b1, long long c1) {
    return total < (1 << 21) ? (long long)((unsigned)a1 * (unsigned)b1 / (unsigned)c1) : a1 * b1 / c1;
  };
  // at least a step per block, so that every block from an item's first to
  // its last has a part of it
  auto cut = [&]() {
    blocks = min((long long)gridDim.x, total);
    begin = share(me, total, blocks);
    end = share(me + 1, total, blocks);
  };
  auto find = [&](int b, int v, long long hi) {
    const long long lo = hi - (long long)v * items;
    if (lo <= begin && begin < hi) {
      sm.start[0] = b;
      // (a sequence's line is below 2^31: at most 2^30 tokens of 32 or more a step, by the heads)
      sm.start[1] = total < (1 << 21) ? (int)((unsigned)(begin - lo) / (unsigned)v) : (int)((begin - lo) / v);
      sm.start[2] = (int)(begin - lo - (long long)sm.start[1] * v);
      sm.start[3] = own_len;
    }
  };
  if (a.batch <= kThreads) {
    const int v = steps_at(tid);
    const int2 s = scan(v);
    total = (long long)s.y * items;
    cut();
    if (me >= blocks) return;
    find(tid, v, (long long)s.x * items);
  } else {
    for (int b0 = 0; b0 < a.batch; b0 += kThreads) total += (long long)scan(steps_at(b0 + tid)).y * items;
    cut();
    if (me >= blocks) return;
    long long carry = 0;
    for (int b0 = 0; b0 < a.batch; b0 += kThreads) {
      const int v = steps_at(b0 + tid);
      const int2 s = scan(v);
      find(b0 + tid, v, carry + (long long)s.x * items);
      carry += (long long)s.y * items;
    }
  }
  __syncthreads();

  Place load;  // what the ring loads next
  load.b = sm.start[0];
  load.item = sm.start[1];
  load.step = sm.start[2];
  load.len = sm.start[3];
  load.steps = steps_of<kStep>(load.len);
  Place cur = load;  // what the products take next
  long long load_left = end - begin, left = end - begin;
  auto next_item = [&](Place& q) {
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
  // A lane copies chunk c of every kLaneRows-th row. The swizzled places of
  // its rows repeat after 8 rows (kPeriod copies), 1 KiB or less apart.
  constexpr int kLaneRows = 32 / kChunks;
  constexpr int kPeriod = kLaneRows >= 8 ? 1 : 8 / kLaneRows;
  const int r0 = lane / kChunks, c0 = lane % kChunks;
  uint32_t place[kPeriod];
#pragma unroll
  for (int i = 0; i < kPeriod; ++i) place[i] = tile_at<kRowBytes>(r0 + i * kLaneRows, c0);
  const uint8_t* const k_lane = static_cast<const uint8_t*>(a.cache.k) + r0 * kRowBytes + c0 * 16;
  const uint8_t* const v_lane = static_cast<const uint8_t*>(a.cache.v) + r0 * kRowBytes + c0 * 16;
  // a 16-byte copy from the cache into the ring
  const uint32_t shared = (uint32_t)__cvta_generic_to_shared(smem_raw);
  const size_t cache_bytes = cache_rows(a.cache) * kRowBytes;
  auto fetch = [&](uint32_t to, const uint8_t* from, const void* cache, bool valid) {
    if (in_smem(to, 16, shared, a.err)) cp16(to, ld_at(from, static_cast<const uint8_t*>(cache), cache_bytes - 15, a.err), valid);
  };
  auto issue = [&](int slot) {  // the next step's tile of this warp into a ring slot
    if (load_left > 0) {
      --load_left;
      const int tok0 = (load.step * kWarps + warp) * kTok;
      if (tok0 < load.len) {
        const int head = load.item / p.tiles;
        const uint32_t dst = ring + slot * (2 * kTileBytes);
        const bool whole = tok0 + kTok <= load.len;
#pragma unroll
        for (int i = 0; i < kPages; ++i) {  // 16 rows in one page
          const int tok = tok0 + 16 * i;
          if (tok < load.len || whole) {
            const size_t at =
                ((((size_t)page_of(a, load.b, tok >> shift) * a.cache.kv_heads + head) << shift) + (tok & mask)) * kRowBytes;
            const uint8_t* k = k_lane + at;
            const uint8_t* v = v_lane + at;
#pragma unroll
            for (int x = 0; x < 16 / kLaneRows; ++x) {
              const int n = i * (16 / kLaneRows) + x;
              const uint32_t to = dst + place[n % kPeriod] + n / kPeriod * kPeriod * kLaneRows * kRowBytes;
              if (whole) {
                fetch(to, k + x * kLaneRows * kRowBytes, a.cache.k, true);
                fetch(to + kTileBytes, v + x * kLaneRows * kRowBytes, a.cache.v, true);
              } else {
                const bool valid = tok + r0 + x * kLaneRows < load.len;
                fetch(to, valid ? k + x * kLaneRows * kRowBytes : k_lane, a.cache.k, valid);
                fetch(to + kTileBytes, valid ? v + x * kLaneRows * kRowBytes : v_lane, a.cache.v, valid);
              }
            }
          } else {  // rows beyond the sequence, as zeros
#pragma unroll
            for (int x = 0; x < 16 / kLaneRows; ++x) {
              const int n = i * (16 / kLaneRows) + x;
              const uint32_t to = dst + place[n % kPeriod] + n / kPeriod * kPeriod * kLaneRows * kRowBytes;
              fetch(to, k_lane, a.cache.k, false);
              fetch(to + kTileBytes, v_lane, a.cache.v, false);
            }
          }
        }
      }
      if (++load.step == load.steps) next_item(load);
    }
    cp_commit();
  };
  // the queries of an item as B fragments, head g of each column block (raw);
  // the next item's are in flight while this one's parts are joined
  uint32_t qf[kNb][D / 16][2];
  auto load_queries = [&](const Place& q) {
    const int head = q.item / p.tiles, head0 = (q.item % p.tiles) * kHeads;
#pragma unroll
    for (int nb = 0; nb < kNb; ++nb) {
      const int h = 8 * nb + g;
      const bool some = h < min(kHeads, p.group - head0);
      const uint16_t* from = a.q + (size_t)q.b * a.ldq + (size_t)(head * p.group + head0 + (some ? h : 0)) * D;
#pragma unroll
      for (int i = 0; i < D / 16; ++i)
#pragma unroll
        for (int w = 0; w < 2; ++w) {
          const int d = k8 ? 16 * i + 4 * t + 2 * w : 16 * i + 2 * t + 8 * w;
          qf[nb][i][w] = some ? *ld_at(reinterpret_cast<const uint32_t*>(from + d), reinterpret_cast<const uint32_t*>(a.q),
                                       span(a.batch, a.ldq, a.heads * D) / 2, a.err)
                              : 0;
        }
    }
  };
  load_queries(cur);
#pragma unroll
  for (int i = 0; i < kSlots - 1; ++i) issue(i);
  int slot = 0;

  while (left > 0) {
    // one item's steps of this run
    const int head = cur.item / p.tiles, head0 = (cur.item % p.tiles) * kHeads;
    const int heads = min(kHeads, p.group - head0);
    const bool starts = cur.step == 0;
    const int n = (int)min((long long)(cur.steps - cur.step), left);
    const bool ends = cur.step + n == cur.steps;

    // For the e4m3 cache the queries are taken in fp16, with the dimensions of
    // a k-step in the order its codes come in (4t, 4t + 1 | 4t + 2, 4t + 3),
    // each head divided by a power of two (dimensions below 2^-15 of the
    // head's largest lose bits to it). mult: of this lane's accumulator
    // columns, heads 2t and 2t + 1.
    float mult[kNb][2];
#pragma unroll
    for (int nb = 0; nb < kNb; ++nb) {
      const float m0 = k8 ? positive(p.mult * *ld_at(a.cache.k_scale + head, a.cache.k_scale, (size_t)a.cache.kv_heads, a.err)) : p.mult;
      float top = 0.f;
#pragma unroll
      for (int i = 0; i < D / 16; ++i)
#pragma unroll
        for (int w = 0; w < 2; ++w) {
          qf[nb][i][w] ^= p.negate;
          if (k8 && kB) {
            const float2 f = unpack16<true>(qf[nb][i][w]);
            top = fmaxf(top, fmaxf(fabsf(f.x), fabsf(f.y)));
          }
        }
      if (k8 && kB) {
        top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 1));
        top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 2));
        // 2^e with |q| 2^-e < 4, from the exponent's bits (e from -126 to 126)
        const int e = min(max((int)(__float_as_uint(top) >> 23), 1), 253);
        const float down = __uint_as_float((uint32_t)(254 - e) << 23), own = positive(m0 * __uint_as_float((uint32_t)e << 23));
#pragma unroll
        for (int i = 0; i < D / 16; ++i)
#pragma unroll
          for (int w = 0; w < 2; ++w) {
            const float2 f = unpack16<true>(qf[nb][i][w]);
            qf[nb][i][w] = pack16<false>(f.x * down, f.y * down);
          }
        mult[nb][0] = __shfl_sync(0xffffffffu, own, 8 * t);
        mult[nb][1] = __shfl_sync(0xffffffffu, own, 8 * t + 4);
      } else {
        mult[nb][0] = mult[nb][1] = m0;
      }
    }

    float o[kNb][D / 16][4];  // dimensions g, g + 8 (k8: 2g, 2g + 1) x heads 2t, 2t + 1
    float m[kNb][2], l[kNb][2];
#pragma unroll
    for (int nb = 0; nb < kNb; ++nb) {
#pragma unroll
      for (int i = 0; i < D / 16; ++i)
#pragma unroll
        for (int j = 0; j < 4; ++j) o[nb][i][j] = 0.f;
      m[nb][0] = m[nb][1] = -INFINITY;
      l[nb][0] = l[nb][1] = 0.f;
    }

    for (int k = 0; k < n; ++k) {
      cp_wait<kSlots - 2>();
      __syncwarp();
      issue(slot == 0 ? kSlots - 1 : slot - 1);  // into the slot read one step ago
      const int tok0 = (cur.step * kWarps + warp) * kTok;
      const uint32_t kt = ring + slot * (2 * kTileBytes), vt = kt + kTileBytes;
      if (tok0 < cur.len) {
        // scores: 16 tokens (g, g + 8) x 8 heads (2t, 2t + 1) at a time
        float s[kTok / 16][kNb][4];
#pragma unroll
        for (int i = 0; i < kTok / 16; ++i)
#pragma unroll
          for (int nb = 0; nb < kNb; ++nb)
#pragma unroll
            for (int j = 0; j < 4; ++j) s[i][nb][j] = 0.f;
#pragma unroll
        for (int c = 0; c < kChunks; c += 2)
#pragma unroll
          for (int i = 0; i < kTok / 16; ++i) {
            // tokens 0-7 and 8-15 of chunk c, then of chunk c + 1
            uint32_t r[4];
            ldsm4(r, kt + tile_at<kRowBytes>(16 * i + (lane & 15), c + (lane >> 4)));
            if (k8) {
#pragma unroll
              for (int x = 0; x < 2; ++x) {
                uint32_t f[4];
                e4m3x4_to_half2x2(r[2 * x], f[0], f[2]);
                e4m3x4_to_half2x2(r[2 * x + 1], f[1], f[3]);
#pragma unroll
                for (int nb = 0; nb < kNb; ++nb) mma<kP>(s[i][nb], f, qf[nb][c + x][0], qf[nb][c + x][1]);
              }
            } else {
#pragma unroll
              for (int nb = 0; nb < kNb; ++nb) mma<kP>(s[i][nb], r, qf[nb][c / 2][0], qf[nb][c / 2][1]);
            }
          }
        if (tok0 + kTok > cur.len) {
#pragma unroll
          for (int i = 0; i < kTok / 16; ++i)
#pragma unroll
            for (int nb = 0; nb < kNb; ++nb)
#pragma unroll
              for (int j = 0; j < 4; ++j)
                if (tok0 + 16 * i + g + 8 * (j >> 1) >= cur.len) s[i][nb][j] = -INFINITY;
        }
        bool grew = false;
        float shift2[kNb][2];
#pragma unroll
        for (int nb = 0; nb < kNb; ++nb)
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            float top = fmaxf(s[0][nb][h], s[0][nb][2 + h]);
#pragma unroll
            for (int i = 1; i < kTok / 16; ++i) top = fmaxf(top, fmaxf(s[i][nb][h], s[i][nb][2 + h]));
            top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 4));
            top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 8));
            top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 16)) * mult[nb][h];
            grew |= top > m[nb][h];
            shift2[nb][h] = fmaxf(m[nb][h], top);
          }
        if (__any_sync(0xffffffffu, grew)) {
#pragma unroll
          for (int nb = 0; nb < kNb; ++nb) {
            float f[2];
#pragma unroll
            for (int h = 0; h < 2; ++h) {
              f[h] = ex2(m[nb][h] - (shift2[nb][h] == -INFINITY ? 0.f : shift2[nb][h]));
              l[nb][h] *= f[h];
              m[nb][h] = shift2[nb][h];
            }
#pragma unroll
            for (int i = 0; i < D / 16; ++i)
#pragma unroll
              for (int j = 0; j < 4; ++j) o[nb][i][j] *= f[j & 1];
          }
        }
        // probabilities, rounded to 16 bits for the product (relative 2^-11
        // or 2^-8 of each term; fp16 has fewer bits for terms below 2^-14 of
        // the warp's maximum and none below 2^-25, while the sum takes them
        // whole), as B fragments: 16 tokens x 8 heads. (A maximum of -inf,
        // where infinite keys leave no score, subtracts 0.)
        float base[kNb][2];
#pragma unroll
        for (int nb = 0; nb < kNb; ++nb)
#pragma unroll
          for (int h = 0; h < 2; ++h) base[nb][h] = m[nb][h] == -INFINITY ? 0.f : -m[nb][h];
        uint32_t pf[kTok / 16][kNb][2];
#pragma unroll
        for (int i = 0; i < kTok / 16; ++i)
#pragma unroll
          for (int nb = 0; nb < kNb; ++nb) {
#pragma unroll
            for (int j = 0; j < 4; ++j) {
              s[i][nb][j] = ex2(fmaf(s[i][nb][j], mult[nb][j & 1], base[nb][j & 1]));
              l[nb][j & 1] += s[i][nb][j];
            }
            pf[i][nb][0] = transpose8(pack16<kP>(s[i][nb][0], s[i][nb][1]));
            pf[i][nb][1] = transpose8(pack16<kP>(s[i][nb][2], s[i][nb][3]));
          }
#pragma unroll
        for (int i = 0; i < kTok / 16; ++i)
#pragma unroll
          for (int c = 0; c < kChunks; c += 2) {
            if (k8) {
              // transposed 16-bit units: tokens 0-7 and 8-15 of chunk c, then
              // of chunk c + 1. A register holds dimensions (2g, 2g + 1) of
              // two tokens: the even ones of both are row g, the odd ones row
              // g + 8
              uint32_t r[4];
              ldsm4t(r, vt + tile_at<kRowBytes>(16 * i + (lane & 15), c + (lane >> 4)));
#pragma unroll
              for (int x = 0; x < 2; ++x) {
                uint32_t f[4];
                e4m3x4_to_half2x2(__byte_perm(r[2 * x], 0, 0x3120), f[0], f[1]);
                e4m3x4_to_half2x2(__byte_perm(r[2 * x + 1], 0, 0x3120), f[2], f[3]);
#pragma unroll
                for (int nb = 0; nb < kNb; ++nb) mma<kP>(o[nb][c + x], f, pf[i][nb][0], pf[i][nb][1]);
              }
            } else {
              // transposed: dimensions 0-7 and 8-15 of the pair of chunks for
              // tokens 0-7, then for tokens 8-15
              uint32_t r[4];
              ldsm4t(r, vt + tile_at<kRowBytes>(16 * i + (lane & 7) + 8 * (lane >> 4), c + ((lane >> 3) & 1)));
#pragma unroll
              for (int nb = 0; nb < kNb; ++nb) mma<kP>(o[nb][c / 2], r, pf[i][nb][0], pf[i][nb][1]);
            }
          }
      }
      slot = slot == kSlots - 1 ? 0 : slot + 1;
      ++cur.step;
    }
    Place next = cur;
    if (left > n) {
      next_item(next);
      load_queries(next);
    }

    // join the warps
#pragma unroll
    for (int nb = 0; nb < kNb; ++nb)
#pragma unroll
      for (int h = 0; h < 2; ++h) {
#pragma unroll
        for (int w = 4; w < 32; w <<= 1) l[nb][h] += __shfl_xor_sync(0xffffffffu, l[nb][h], w);
        if (g == 0) {
          sm.ml[0][warp][8 * nb + 2 * t + h] = m[nb][h];
          sm.ml[1][warp][8 * nb + 2 * t + h] = l[nb][h];
        }
      }
    __syncthreads();
    if (tid < kHeads) {
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
    __syncthreads();
    const bool whole = starts && ends;
    float* part = p.parts + (size_t)(2 * me + (starts ? 1 : 0)) * kPartFloats<D, kHeads>;
    const float v_scale = k8 ? *ld_at(a.cache.v_scale + head, a.cache.v_scale, (size_t)a.cache.kv_heads, a.err) : 1.f;
    const size_t out0 = (size_t)cur.b * a.heads + head * p.group + head0;
    auto put_out = [&](int h, int d, uint2 v) {
      uint16_t* to = a.out + (out0 + h) * D + d;
      if (in_buf(to, a.out, (size_t)a.batch * a.heads * D - 3, a.err)) *reinterpret_cast<uint2*>(to) = v;
    };
    auto put_lse = [&](int h, float top, float sum) {
      if (a.lse && in_buf(a.lse + out0 + h, a.lse, (size_t)a.batch * a.heads, a.err))
        a.lse[out0 + h] = sum == 0.f ? -INFINITY : top * kLn2 + logf(sum);
    };
#pragma unroll
    for (int nb = 0; nb < kNb; ++nb)
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const float top = sm.top[8 * nb + 2 * t + h];
        const float f = ex2(m[nb][h] - (top == -INFINITY ? 0.f : top));
#pragma unroll
        for (int i = 0; i < D / 16; ++i) o[nb][i][h] *= f, o[nb][i][2 + h] *= f;
      }
#pragma unroll
    for (int round = 0; round < kHeads / kJoinHeads; ++round) {
      if (round * kJoinHeads >= heads) break;
      if (round) __syncthreads();  // the heads before these are read
      if ((t >> 1) == (round & 1)) {
        const int nb = round >> 1;
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          const int r = 2 * (t & 1) + h;  // of the round's heads
          float* row = &sm.o[warp][r][0];
#pragma unroll
          for (int i = 0; i < D / 16; ++i) {
            if (k8) {
              *reinterpret_cast<float2*>(row + join_at(r, 16 * i + 2 * g)) = make_float2(o[nb][i][h], o[nb][i][2 + h]);
            } else {
              row[join_at(r, 16 * i + g)] = o[nb][i][h];
              row[join_at(r, 16 * i + 8 + g)] = o[nb][i][2 + h];
            }
          }
        }
      }
      __syncthreads();
      const int some = min(kJoinHeads, heads - round * kJoinHeads);
      for (int u = tid; u < some * (D / 4); u += kThreads) {
        const int r = u / (D / 4), d = u % (D / 4) * 4, h = round * kJoinHeads + r;
        float4 v = *reinterpret_cast<const float4*>(&sm.o[0][r][join_at(r, d)]);
#pragma unroll
        for (int w = 1; w < kWarps; ++w) {
          const float4 x = *reinterpret_cast<const float4*>(&sm.o[w][r][join_at(r, d)]);
          v.x += x.x, v.y += x.y, v.z += x.z, v.w += x.w;
        }
        if (whole) {
          const float l1 = sm.sum[h], inv = l1 == 0.f ? 0.f : v_scale / l1;  // (a NaN sum is the result)
          put_out(h, d, make_uint2(pack16<kB>(v.x * inv, v.y * inv), pack16<kB>(v.z * inv, v.w * inv)));
        } else if (in_buf(part + h * D + d, p.parts, p.part_floats - 3, a.err)) {
          *reinterpret_cast<float4*>(part + h * D + d) = v;
        }
      }
    }
    if (tid < heads) {
      if (whole) {
        put_lse(tid, sm.top[tid], sm.sum[tid]);
      } else if (in_buf(part + kHeads * D + kHeads + tid, p.parts, p.part_floats, a.err)) {
        part[kHeads * D + tid] = sm.top[tid];
        part[kHeads * D + kHeads + tid] = sm.sum[tid];
      }
    }

    if (!whole) {
      // this item's steps in the line, and the blocks that have a part of it
      const long long at = begin + (end - begin - left) - (cur.step - n);  // the item's first step
      // (block c holds the steps from floor(c total / blocks) on)
      auto holder = [&](long long step) {
        const long long x = (step + 1) * blocks - 1;
        return total < (1 << 21) ? (long long)((unsigned)x / (unsigned)total) : x / total;
      };
      const long long first = holder(at), final = holder(at + cur.steps - 1);
      __syncthreads();
      if (tid == 0) {
        // the block's part before its arrival, the others' before what follows
        int before = -1;
        if (in_buf(p.arrived + first, p.arrived, kFlagBytes / sizeof(int), a.err))
          asm volatile("atom.add.acq_rel.gpu.global.s32 %0, [%1], 1;" : "=r"(before) : "l"(p.arrived + first) : "memory");
        sm.last = before == (int)(final - first);
      }
      __syncthreads();
      if (sm.last) {
        const int count = (int)(final - first) + 1;
        // four dimensions of a head per thread, kBatch parts in flight: their
        // maxima, sums and values arrive in one round of latency
        constexpr int kBatch = 8;
        for (int u = tid; u < heads * (D / 4); u += kThreads) {
          const int h = u / (D / 4), d = u % (D / 4) * 4;
          float top = -INFINITY, sum = 0.f;
          float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
          for (int i0 = 0; i0 < count; i0 += kBatch) {
            float mi[kBatch], li[kBatch];
            float4 x[kBatch];
#pragma unroll
            for (int i = 0; i < kBatch; ++i) {
              mi[i] = -INFINITY, li[i] = 0.f;
              x[i] = make_float4(0.f, 0.f, 0.f, 0.f);
              if (i0 + i < count) {
                const float* q = p.parts + (size_t)(2 * (first + i0 + i) + (i0 + i == 0 ? 1 : 0)) * kPartFloats<D, kHeads>;
                q = ld_at(q, p.parts, p.part_floats - kPartFloats<D, kHeads> + 1, a.err);
                mi[i] = __ldcg(q + kHeads * D + h);
                li[i] = __ldcg(q + kHeads * D + kHeads + h);
                x[i] = __ldcg(reinterpret_cast<const float4*>(q + h * D + d));
              }
            }
            float now = top;
#pragma unroll
            for (int i = 0; i < kBatch; ++i) now = fmaxf(now, mi[i]);
            const float base = now == -INFINITY ? 0.f : now;
            const float old = ex2(top - base);
            top = now;
            sum *= old, v.x *= old, v.y *= old, v.z *= old, v.w *= old;
#pragma unroll
            for (int i = 0; i < kBatch; ++i) {
              const float f = ex2(mi[i] - base);
              sum = fmaf(li[i], f, sum);
              v.x = fmaf(x[i].x, f, v.x), v.y = fmaf(x[i].y, f, v.y), v.z = fmaf(x[i].z, f, v.z), v.w = fmaf(x[i].w, f, v.w);
            }
          }
          const float inv = sum == 0.f ? 0.f : v_scale / sum;
          put_out(h, d, make_uint2(pack16<kB>(v.x * inv, v.y * inv), pack16<kB>(v.z * inv, v.w * inv)));
          if (d == 0) put_lse(h, top, sum);
        }
        if (tid == 0) p.arrived[first] = 0;  // left zero for the next call
      }
    }
    left -= n;
    cur = next;
    __syncthreads();  // the shared maxima and rows are free again
  }
  cp_wait<0>();
}

template <bool kB, bool k8, int D, int kHeads>
cudaError_t launch(const DecodeArgs& p, int sms, cudaStream_t stream) {
  auto kern = attn_decode_kernel<kB, k8, D, kHeads>;
  cudaError_t e = set_max_smem_once(reinterpret_cast<const void*>(kern), (int)sizeof(Smem<D, kHeads>));
  if (e != cudaSuccess) return e;
  // no more blocks than there can be steps (a block without one costs its
  // launch: 1 x 777, 104 steps, 8.0 us with 104 blocks, 8.2 with all 456)
  constexpr int kStep = kWarps * kTileBytes / (D * (k8 ? 1 : 2));
  const long long longest = (((long long)p.a.max_pages << p.a.cache.page_shift) + kStep - 1) / kStep;
  const long long steps = (longest > 0 ? longest : 1) * p.a.batch * p.a.cache.kv_heads * p.tiles;
  const long long most = (long long)kBlocks<kHeads> * sms;
  return launch_pdl(kern, dim3((unsigned)(steps < most ? steps : most)), dim3(kThreads), sizeof(Smem<D, kHeads>), stream, p);
}

template <bool kB, bool k8, int D>
cudaError_t launch_heads(DecodeArgs& p, int sms, cudaStream_t stream) {
  const int heads = p.group <= 8 ? 8 : 16;
  p.tiles = (p.group + heads - 1) / heads;
  return heads == 8 ? launch<kB, k8, D, 8>(p, sms, stream) : launch<kB, k8, D, 16>(p, sms, stream);
}

}  // namespace

size_t attn_decode_workspace_bytes(int head_dim, int sms) {
  const size_t few = (size_t)kBlocks<8> * 8, many = (size_t)kBlocks<16> * 16;  // heads of an SM's parts
  return kFlagBytes + (size_t)sms * 2 * (few > many ? few : many) * (head_dim + 2) * sizeof(float);
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
  p.part_floats = (attn_decode_workspace_bytes(head_dim, sms) - kFlagBytes) / sizeof(float);
  p.group = args.heads / args.cache.kv_heads;
  // the scores' maximum is taken before the scale, so it has to be positive:
  // a negative scale negates the queries, and a scale of zero becomes one too
  // small to tell from it
  p.mult = fmaxf(fabsf(args.scale) * kLog2e, 1e-37f);
  p.negate = args.scale < 0.f ? 0x80008000u : 0u;
  switch ((bf16 ? 4 : 0) | (e4m3 ? 2 : 0) | (head_dim == 128 ? 1 : 0)) {
    case 0: return launch_heads<false, false, 64>(p, sms, stream);
    case 1: return launch_heads<false, false, 128>(p, sms, stream);
    case 2: return launch_heads<false, true, 64>(p, sms, stream);
    case 3: return launch_heads<false, true, 128>(p, sms, stream);
    case 4: return launch_heads<true, false, 64>(p, sms, stream);
    case 5: return launch_heads<true, false, 128>(p, sms, stream);
    case 6: return launch_heads<true, true, 64>(p, sms, stream);
    default: return launch_heads<true, true, 128>(p, sms, stream);
  }
}

}  // namespace w4a16
