// C ABI of the decoder layer's other operators: argument checks and launches.
// Declarations and the contract of every entry point: include/w4a16.h.
#include <cmath>
#include <cstdarg>
#include <cstdio>

#include "common.cuh"
#include "experts.cuh"
#include "kernels.h"
#include "layer.cuh"

namespace w4a16 {
namespace {

int fail(int code, const char* fmt, ...) {
  char buf[512];
  va_list ap;
  va_start(ap, fmt);
  vsnprintf(buf, sizeof(buf), fmt, ap);
  va_end(ap);
  return report_error(code, buf);
}

int finish(cudaError_t e, const char* what) {
  if (e == cudaSuccess) return report_ok();
  return fail(W4A16_ERR_CUDA, "%s: %s (%s)", what, cudaGetErrorName(e), cudaGetErrorString(e));
}

bool aligned(const void* p, size_t a) { return (reinterpret_cast<uintptr_t>(p) % a) == 0; }

constexpr int kMaxRows = 1 << 20, kMaxHeads = 1024, kMaxTokens = 1 << 30;

// The rules of the paged cache that the append and the attention share.
int check_cache(const void* k, const void* v, const float* k_scale, const float* v_scale, int pages, int page_size,
                int heads, int kv_heads, int head_dim, int flags, int* page_shift) {
  if (heads <= 0 || kv_heads <= 0) return fail(W4A16_ERR_INVALID_ARG, "heads=%d, kv_heads=%d must be positive", heads, kv_heads);
  if (pages <= 0 || page_size <= 0) return fail(W4A16_ERR_INVALID_ARG, "pages=%d, page_size=%d must be positive", pages, page_size);
  if (heads > kMaxHeads || heads % kv_heads)
    return fail(W4A16_ERR_UNSUPPORTED_SHAPE, "heads=%d is above %d or no multiple of kv_heads=%d", heads, kMaxHeads, kv_heads);
  if (head_dim != 64 && head_dim != 128) return fail(W4A16_ERR_UNSUPPORTED_SHAPE, "head_dim=%d is neither 64 nor 128", head_dim);
  if (page_size < 16 || page_size > 256 || (page_size & (page_size - 1)))
    return fail(W4A16_ERR_UNSUPPORTED_SHAPE, "page_size=%d is not 16, 32, 64, 128 or 256", page_size);
  if ((long long)pages * kv_heads * page_size > 0x7fffffffll)
    return fail(W4A16_ERR_UNSUPPORTED_SHAPE, "%d pages of %d x %d rows: a cache of 2^31 rows or more", pages, kv_heads, page_size);
  if (!k || !v) return fail(W4A16_ERR_INVALID_ARG, "null cache pointer");
  if (!aligned(k, 16) || !aligned(v, 16)) return fail(W4A16_ERR_MISALIGNED, "alignment: the caches need 16 bytes");
  const bool e4m3 = (flags & W4A16_CACHE_E4M3) != 0;
  if (e4m3 && (!k_scale || !v_scale)) return fail(W4A16_ERR_INVALID_ARG, "an e4m3 cache needs k_scale and v_scale");
  if (!e4m3 && (k_scale || v_scale)) return fail(W4A16_ERR_INVALID_ARG, "scales go with an e4m3 cache only");
  if (!aligned(k_scale, 4) || !aligned(v_scale, 4)) return fail(W4A16_ERR_MISALIGNED, "alignment: the scales need 4 bytes");
  int s = 4;
  while ((1 << s) < page_size) ++s;
  *page_shift = s;
  return W4A16_OK;
}

// Checks shared by the two attention entry points; fills the kernel's
// arguments.
int check_attn(AttnArgs* a, const uint16_t* q, int64_t q_stride, const void* k, const void* v, const float* k_scale,
               const float* v_scale, int pages, int page_size, const int32_t* table, int64_t table_stride,
               int max_pages, const int32_t* lens, int rows, int batch, int heads, int kv_heads, int head_dim,
               float scale, uint16_t* out, float* lse, int flags) {
  if (rows < 0 || batch < 0) return fail(W4A16_ERR_INVALID_ARG, "tokens=%d, batch=%d: negative", rows, batch);
  if (flags & ~(W4A16_BF16 | W4A16_CACHE_E4M3)) return fail(W4A16_ERR_INVALID_ARG, "flags=0x%x: unknown bits", flags);
  int shift = 0;
  if (int rc = check_cache(k, v, k_scale, v_scale, pages, page_size, heads, kv_heads, head_dim, flags, &shift)) return rc;
  if (rows > kMaxRows || batch > kMaxRows)
    return fail(W4A16_ERR_UNSUPPORTED_SHAPE, "tokens=%d or batch=%d above %d", rows, batch, kMaxRows);
  if (max_pages < 0 || table_stride < max_pages)
    return fail(W4A16_ERR_INVALID_ARG, "max_pages=%d is negative or above the table's row stride", max_pages);
  if ((long long)max_pages << shift > kMaxTokens)
    return fail(W4A16_ERR_UNSUPPORTED_SHAPE, "%d pages of %d tokens per sequence: above 2^30 tokens", max_pages, page_size);
  if (!std::isfinite(scale)) return fail(W4A16_ERR_INVALID_ARG, "scale=%g is not finite", (double)scale);
  if (q_stride < (int64_t)heads * head_dim) return fail(W4A16_ERR_INVALID_ARG, "q's row stride is below heads * head_dim");
  // (no sequence has no lengths, and sequences of no pages have no table)
  if (rows > 0 && batch > 0 && (!q || (!table && max_pages > 0) || !lens || !out)) return fail(W4A16_ERR_INVALID_ARG, "null pointer");
  if (!aligned(q, 16) || !aligned(out, 16) || q_stride % 8)
    return fail(W4A16_ERR_MISALIGNED, "alignment: q, its rows and out need 16 bytes");
  if (!aligned(table, 4) || !aligned(lens, 4) || !aligned(lse, 4))
    return fail(W4A16_ERR_MISALIGNED, "alignment: table, lens and lse need 4 bytes");
  a->q = q;
  a->ldq = q_stride;
  a->cache = {k, v, k_scale, v_scale, pages, shift, kv_heads};
  a->table = table;
  a->table_ld = table_stride;
  a->max_pages = max_pages;
  a->starts = nullptr;
  a->lens = lens;
  a->rows = rows;
  a->batch = batch;
  a->heads = heads;
  a->scale = scale;
  a->out = out;
  a->lse = lse;
  a->err = nullptr;
  return W4A16_OK;
}

int check_workspace(const void* workspace, size_t bytes, size_t need) {
  if (need > 0 && (!workspace || bytes < need))
    return fail(W4A16_ERR_WORKSPACE_TOO_SMALL, "the call needs a workspace of %zu bytes (got %zu)", need,
                workspace ? bytes : (size_t)0);
  if (need > 0 && !aligned(workspace, 256)) return fail(W4A16_ERR_MISALIGNED, "workspace needs 256-byte alignment");
  return W4A16_OK;
}

constexpr int kMaxExperts = 512, kMaxTop = 32;

int check_routing(int T, int E, int top_k) {
  if (T < 0 || E <= 0 || top_k <= 0)
    return fail(W4A16_ERR_INVALID_ARG, "T=%d is negative, or E=%d or top_k=%d not positive", T, E, top_k);
  if (T > kMaxRows || E > kMaxExperts || top_k > kMaxTop || top_k > E)
    return fail(W4A16_ERR_UNSUPPORTED_SHAPE, "T=%d above %d, E=%d above %d, or top_k=%d above %d or E", T, kMaxRows, E,
                kMaxExperts, top_k, kMaxTop);
  return W4A16_OK;
}

// The path, the shape rules and the flags of the products grouped by expert.
int check_experts(int T, int top_k, int E, int N, int K, int group, int flags) {
  if (int rc = check_routing(T, E, top_k)) return rc;
  constexpr int known = W4A16_BF16 | W4A16_SILU_MUL | W4A16_EXPERTS_PER_CHOICE | W4A16_EXPERTS_COMBINE;
  const int path = flags & 0xff;
  if ((flags & ~(known | 0xff)) || (path != W4A16_PATH_AUTO && path != W4A16_PATH_DECODE && path != W4A16_PATH_TENSOR_PAIR))
    return fail(W4A16_ERR_INVALID_ARG, "flags=0x%x: unknown bits or path", flags);
  if ((flags & W4A16_SILU_MUL) && (flags & W4A16_EXPERTS_COMBINE))
    return fail(W4A16_ERR_INVALID_ARG, "W4A16_SILU_MUL does not go with W4A16_EXPERTS_COMBINE");
  if (N <= 0 || K <= 0 || group <= 0) return fail(W4A16_ERR_INVALID_ARG, "N=%d, K=%d, group=%d must be positive", N, K, group);
  if (N > kMaxRows || K > kMaxRows || N % 16 || K % 64 || group % 64 || K % group)
    return fail(W4A16_ERR_UNSUPPORTED_SHAPE, "N=%d, K=%d, group=%d: N %% 16, K %% 64, group %% 64 and K %% group must be 0", N, K, group);
  if ((flags & W4A16_SILU_MUL) && N % 32)
    return fail(W4A16_ERR_UNSUPPORTED_SHAPE, "N=%d: gate and up need a multiple of 32", N);
  if ((long long)E * N > 0x7fffffffll) return fail(W4A16_ERR_UNSUPPORTED_SHAPE, "E=%d experts of N=%d columns: above 2^31", E, N);
  return W4A16_OK;
}

// Whether a call takes the kernel on the tensor cores: above 24 rows per expert
// on average. Measured (us, few rows against tensor cores): 64 experts of 2048 x
// 2048, top 8, 16 rows each 64 against 84, 24 86 against 85, 32 107 against 85; 8
// of 4096 x 22016, top 2, 24 193 against 199, 32 256 against 199; 8 of 11008 x
// 4096, 24 123 against 108; 128 of 4096 x 3584, top 8, 16 384 against 477, 24 516
// against 460.
bool experts_on_tensor_cores(int T, int top_k, int E, int flags) {
  const int path = flags & 0xff;
  if (path != W4A16_PATH_AUTO) return path == W4A16_PATH_TENSOR_PAIR;
  return (long long)T * top_k > 24ll * E;
}

size_t experts_workspace(int T, int top_k, int E, int N, int flags) {
  const bool combine = (flags & W4A16_EXPERTS_COMBINE) != 0;
  if (T == 0) return 0;
  return experts_on_tensor_cores(T, top_k, E, flags) ? experts_tc_workspace_bytes(T * top_k, N, combine)
                                                     : experts_decode_workspace_bytes(T * top_k, N, combine);
}

}  // namespace
}  // namespace w4a16

using namespace w4a16;

extern "C" {

int w4a16_rms_norm(const uint16_t* x, int64_t x_stride, const uint16_t* residual, int64_t residual_stride,
                   const uint16_t* weight, int M, int K, float eps, int flags, uint16_t* y, uint16_t* codes,
                   int8_t* aq, float* s_a, uint16_t* h, int64_t h_stride, void* stream) {
  if (M < 0 || K <= 0) return fail(W4A16_ERR_INVALID_ARG, "M=%d is negative or K=%d not positive", M, K);
  if (flags & ~W4A16_BF16) return fail(W4A16_ERR_INVALID_ARG, "flags=0x%x: only W4A16_BF16", flags);
  if (M > kMaxRows || K > 65536) return fail(W4A16_ERR_UNSUPPORTED_SHAPE, "M=%d above %d or K=%d above 65536", M, kMaxRows, K);
  if (!(eps >= 0.f) || !std::isfinite(eps)) return fail(W4A16_ERR_INVALID_ARG, "eps=%g is negative or not finite", (double)eps);
  if (M == 0) return report_ok();
  if (!x || !weight || (!y && !codes && !aq && !h)) return fail(W4A16_ERR_INVALID_ARG, "null pointer");
  if ((codes || aq) ? !s_a : s_a != nullptr) return fail(W4A16_ERR_INVALID_ARG, "s_a goes with codes or aq");
  if (x_stride < K || (residual && residual_stride < K) || (h && h_stride < K))
    return fail(W4A16_ERR_INVALID_ARG, "a row stride is below K=%d", K);
  if (!aligned(x, 2) || !aligned(residual, 2) || !aligned(weight, 2) || !aligned(y, 2) || !aligned(codes, 2) ||
      !aligned(h, 2) || !aligned(s_a, 4))
    return fail(W4A16_ERR_MISALIGNED, "alignment: 16-bit arrays need 2 bytes, s_a 4");
  return finish(launch_rms_norm(x, x_stride, residual, residual ? residual_stride : 0, weight, M, K, eps,
                                (flags & W4A16_BF16) != 0, y, codes, aq, s_a, h, h ? h_stride : 0, (cudaStream_t)stream),
                "norm launch");
}

int w4a16_rope_append_norm(const uint16_t* qkv, int64_t qkv_stride, const float* cos_sin, int table_len, int rotary,
                           const int32_t* positions, const int64_t* slots, int tokens, int heads, int kv_heads,
                           int head_dim, uint16_t* q, void* k_cache, void* v_cache, const float* k_scale,
                           const float* v_scale, int pages, int page_size, const uint16_t* q_norm,
                           const uint16_t* k_norm, float eps, int flags, void* stream) {
  if (tokens < 0) return fail(W4A16_ERR_INVALID_ARG, "tokens=%d is negative", tokens);
  if (flags & ~(W4A16_BF16 | W4A16_CACHE_E4M3 | W4A16_ROPE_INTERLEAVED))
    return fail(W4A16_ERR_INVALID_ARG, "flags=0x%x: unknown bits", flags);
  int shift = 0;
  if (int rc = check_cache(k_cache, v_cache, k_scale, v_scale, pages, page_size, heads, kv_heads, head_dim, flags, &shift))
    return rc;
  if (tokens > kMaxRows) return fail(W4A16_ERR_UNSUPPORTED_SHAPE, "tokens=%d above %d", tokens, kMaxRows);
  if (rotary < 2 || rotary % 2 || rotary > head_dim)
    return fail(W4A16_ERR_UNSUPPORTED_SHAPE, "rotary=%d is not even and within 2..head_dim=%d", rotary, head_dim);
  if (table_len <= 0) return fail(W4A16_ERR_INVALID_ARG, "table_len=%d must be positive", table_len);
  if (qkv_stride < (int64_t)(heads + 2 * kv_heads) * head_dim)
    return fail(W4A16_ERR_INVALID_ARG, "qkv's row stride is below (heads + 2 kv_heads) * head_dim");
  if (!(eps >= 0.f) || !std::isfinite(eps)) return fail(W4A16_ERR_INVALID_ARG, "eps=%g is negative or not finite", (double)eps);
  if (tokens == 0) return report_ok();
  if (!qkv || !cos_sin || !positions || !slots || !q) return fail(W4A16_ERR_INVALID_ARG, "null pointer");
  if (!aligned(qkv, 2) || !aligned(q, 2) || !aligned(cos_sin, 4) || !aligned(positions, 4) || !aligned(slots, 8) ||
      !aligned(q_norm, 2) || !aligned(k_norm, 2))
    return fail(W4A16_ERR_MISALIGNED, "alignment: qkv, q and the norms need 2 bytes, cos_sin, positions 4, slots 8");
  return finish(launch_rope_append(qkv, qkv_stride, cos_sin, table_len, rotary, positions, slots, tokens, heads,
                                   kv_heads, head_dim, q, k_cache, v_cache, k_scale, v_scale, pages, shift, q_norm, k_norm,
                                   eps, (flags & W4A16_BF16) != 0, (flags & W4A16_CACHE_E4M3) != 0,
                                   (flags & W4A16_ROPE_INTERLEAVED) != 0, (cudaStream_t)stream),
                "rotation and append launch");
}

int w4a16_rope_append(const uint16_t* qkv, int64_t qkv_stride, const float* cos_sin, int table_len, int rotary,
                      const int32_t* positions, const int64_t* slots, int tokens, int heads, int kv_heads,
                      int head_dim, uint16_t* q, void* k_cache, void* v_cache, const float* k_scale,
                      const float* v_scale, int pages, int page_size, int flags, void* stream) {
  return w4a16_rope_append_norm(qkv, qkv_stride, cos_sin, table_len, rotary, positions, slots, tokens, heads, kv_heads,
                                head_dim, q, k_cache, v_cache, k_scale, v_scale, pages, page_size, nullptr, nullptr, 0.f,
                                flags, stream);
}

int w4a16_attn_workspace_size(int tokens, int batch, int heads, int kv_heads, int head_dim, size_t* bytes) {
  if (tokens < 0 || batch < 0 || heads <= 0 || kv_heads <= 0 || head_dim <= 0)
    return fail(W4A16_ERR_INVALID_ARG, "negative or zero size");
  if (!bytes) return fail(W4A16_ERR_INVALID_ARG, "null output pointer");
  *bytes = 0;
  if (tokens == 0 || batch == 0) return report_ok();
  const int sms = device_sms();
  const size_t decode = tokens == batch ? attn_decode_workspace_bytes(head_dim, sms) : 0;
  const size_t prompt = attn_prompt_workspace_bytes(tokens, (heads + kv_heads - 1) / kv_heads, kv_heads, head_dim, sms);
  *bytes = decode > prompt ? decode : prompt;
  return report_ok();
}

int w4a16_attn_decode(const uint16_t* q, int64_t q_stride, const void* k_cache, const void* v_cache,
                      const float* k_scale, const float* v_scale, int pages, int page_size, const int32_t* table,
                      int64_t table_stride, int max_pages, const int32_t* lens, int batch, int heads, int kv_heads,
                      int head_dim, float scale, uint16_t* out, float* lse, void* workspace, size_t workspace_bytes,
                      int flags, void* stream) {
  AttnArgs a;
  if (int rc = check_attn(&a, q, q_stride, k_cache, v_cache, k_scale, v_scale, pages, page_size, table, table_stride,
                          max_pages, lens, batch, batch, heads, kv_heads, head_dim, scale, out, lse, flags))
    return rc;
  if (batch == 0) return report_ok();
  const int sms = device_sms();
  if (int rc = check_workspace(workspace, workspace_bytes, attn_decode_workspace_bytes(head_dim, sms))) return rc;
  return finish(launch_attn_decode(a, head_dim, (flags & W4A16_BF16) != 0, (flags & W4A16_CACHE_E4M3) != 0, workspace,
                                   sms, (cudaStream_t)stream),
                "decode attention launch");
}

int w4a16_attn_prompt(const uint16_t* q, int64_t q_stride, const void* k_cache, const void* v_cache,
                      const float* k_scale, const float* v_scale, int pages, int page_size, const int32_t* table,
                      int64_t table_stride, int max_pages, const int32_t* starts, const int32_t* lens, int tokens,
                      int batch, int heads, int kv_heads, int head_dim, float scale, uint16_t* out, float* lse,
                      void* workspace, size_t workspace_bytes, int flags, void* stream) {
  AttnArgs a;
  if (int rc = check_attn(&a, q, q_stride, k_cache, v_cache, k_scale, v_scale, pages, page_size, table, table_stride,
                          max_pages, lens, tokens, batch, heads, kv_heads, head_dim, scale, out, lse, flags))
    return rc;
  if (tokens == 0 || batch == 0) return report_ok();
  if (!starts) return fail(W4A16_ERR_INVALID_ARG, "null pointer (starts)");
  if (!aligned(starts, 4)) return fail(W4A16_ERR_MISALIGNED, "alignment: starts needs 4 bytes");
  a.starts = starts;
  const int sms = device_sms();
  if (int rc = check_workspace(workspace, workspace_bytes, attn_prompt_workspace_bytes(tokens, heads / kv_heads, kv_heads, head_dim, sms))) return rc;
  return finish(launch_attn_prompt(a, head_dim, (flags & W4A16_BF16) != 0, (flags & W4A16_CACHE_E4M3) != 0, workspace,
                                   sms, (cudaStream_t)stream),
                "prompt attention launch");
}

int w4a16_route_workspace_size(int T, int E, int top_k, size_t* bytes) {
  if (int rc = check_routing(T, E, top_k)) return rc;
  if (!bytes) return fail(W4A16_ERR_INVALID_ARG, "null output pointer");
  *bytes = route_workspace_bytes(T, E);
  return report_ok();
}

int w4a16_route(const void* logits, int64_t logits_stride, int T, int E, int top_k, int32_t* experts, float* weights,
                int32_t* rows, int32_t* offsets, void* workspace, size_t workspace_bytes, int flags, void* stream) {
  if (int rc = check_routing(T, E, top_k)) return rc;
  constexpr int known = W4A16_BF16 | W4A16_ROUTE_FP32 | W4A16_ROUTE_SIGMOID | W4A16_ROUTE_RENORMALIZE;
  if ((flags & ~known) || ((flags & W4A16_BF16) && (flags & W4A16_ROUTE_FP32)))
    return fail(W4A16_ERR_INVALID_ARG, "flags=0x%x: unknown bits, or two types", flags);
  if (logits_stride < E) return fail(W4A16_ERR_INVALID_ARG, "the logits' row stride is below E=%d", E);
  if (!offsets || (T > 0 && (!logits || !experts || !weights || !rows))) return fail(W4A16_ERR_INVALID_ARG, "null pointer");
  const int type = (flags & W4A16_ROUTE_FP32) ? 2 : (flags & W4A16_BF16) ? 1 : 0;
  if (!aligned(logits, type == 2 ? 4 : 2) || !aligned(experts, 4) || !aligned(weights, 4) || !aligned(rows, 4) || !aligned(offsets, 4))
    return fail(W4A16_ERR_MISALIGNED, "alignment: logits need their type's, the results 4 bytes");
  if (int rc = check_workspace(workspace, workspace_bytes, route_workspace_bytes(T, E))) return rc;
  return finish(launch_route(logits, logits_stride, type, T, E, top_k, (flags & W4A16_ROUTE_SIGMOID) != 0,
                             (flags & W4A16_ROUTE_RENORMALIZE) != 0, experts, weights, rows, offsets, workspace,
                             (cudaStream_t)stream),
                "router launch");
}

int w4a16_experts_workspace_size(int T, int top_k, int E, int N, int K, int group, int flags, size_t* bytes) {
  if (int rc = check_experts(T, top_k, E, N, K, group, flags)) return rc;
  if (!bytes) return fail(W4A16_ERR_INVALID_ARG, "null output pointer");
  *bytes = experts_workspace(T, top_k, E, N, flags);
  return report_ok();
}

int w4a16_gemm_experts(const uint16_t* A, const uint32_t* Wq, const uint16_t* scales, const uint32_t* zeros, int T,
                       int top_k, int E, int N, int K, int group, const int32_t* experts, const float* weights,
                       const int32_t* rows, const int32_t* offsets, uint16_t* Y, void* workspace,
                       size_t workspace_bytes, int flags, void* stream) {
  if (int rc = check_experts(T, top_k, E, N, K, group, flags)) return rc;
  if (T == 0) return report_ok();
  const bool combine = (flags & W4A16_EXPERTS_COMBINE) != 0;
  if (!A || !Wq || !scales || !zeros || !experts || !rows || !offsets || !Y || (combine && !weights))
    return fail(W4A16_ERR_INVALID_ARG, "null pointer");
  if (!aligned(A, 16) || !aligned(Wq, 16) || !aligned(scales, 16) || !aligned(Y, 16) || !aligned(zeros, 8) ||
      !aligned(experts, 4) || !aligned(weights, 4) || !aligned(rows, 4) || !aligned(offsets, 4))
    return fail(W4A16_ERR_MISALIGNED, "alignment: A, Wq, scales and Y need 16 bytes, zeros 8, the routing 4");
  const size_t need = experts_workspace(T, top_k, E, N, flags);
  if (int rc = check_workspace(workspace, workspace_bytes, need)) return rc;
  const ExpertArgs a = {A, Wq, scales, zeros, experts, weights, rows, offsets, Y, T, top_k, E, N, K, group,
                        (flags & W4A16_EXPERTS_PER_CHOICE) != 0, (flags & W4A16_SILU_MUL) != 0, combine, nullptr};
  const auto launch = experts_on_tensor_cores(T, top_k, E, flags) ? launch_experts_tc : launch_experts_decode;
  return finish(launch(a, (flags & W4A16_BF16) != 0, need ? workspace : nullptr, (cudaStream_t)stream), "experts' product launch");
}

}  // extern "C"
