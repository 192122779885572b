// Attention over the 8-bit paged KV cache (decode and prefill), with a sliding
// window and first tokens that stay visible.
#include <math.h>

#include "kv8.cuh"

namespace qw {
namespace kv8 {

constexpr float kLog2e = 1.4426950408889634f;

// Error word of this file's kernels: kErrContextOverflow (common.cuh), else a bounded wait that gave up.
__device__ unsigned int g_kv8_error = 0;

// One warp per (query token, q head); lane owns dims 4 lane .. + 3.
template <int KV>
__global__ void __launch_bounds__(128) attn_kv8_kernel(const bf16* __restrict__ q, const Cache c,
                                                       const int32_t* __restrict__ cu_q,
                                                       const int32_t* __restrict__ ctx, int n_seqs, int max_q, int nh,
                                                       int nkv, int max_ctx, float scale_log2, int window,
                                                       int n_sink, bf16* __restrict__ out) {
  pdl_wait();      // inputs of this kernel are complete and visible
  pdl_trigger();   // only now may the next kernel start its prologue
  const int64_t w = (int64_t(blockIdx.x) * blockDim.x + threadIdx.x) >> 5;
  const int lane = threadIdx.x & 31;
  if (w >= int64_t(n_seqs) * max_q * nh) return;
  const int s = int(w / (int64_t(max_q) * nh)), i = int((w / nh) % max_q), h = int(w % nh);
  const int t0 = cu_q != nullptr ? cu_q[s] : s, lq = cu_q != nullptr ? cu_q[s + 1] - t0 : 1;
  if (i >= lq) return;
  const int p = ctx[s] - lq + i;   // key position of this query
  const int g = h / (nh / nkv);
  const int64_t at = (int64_t(t0 + i) * nh + h) * HD + 4 * lane;
  float qv[4], o[4] = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
  for (int e = 0; e < 4; ++e) qv[e] = to_f(q[at + e]);
  float m = -INFINITY, l = 0.0f;
  const int lo = window > 0 ? max(p + 1 - window, 0) : 0;
  if (ctx[s] > max_ctx && lane == 0) atomicOr(&g_kv8_error, kErrContextOverflow);
  const int last = min(p, max_ctx - 1);
  for (int j = 0; j <= last; ++j) {
    if (j < lo && j >= n_sink) j = lo;
    if (j > last) break;
    const int64_t row = row_of(c.table, c.max_blocks, c.block_size, c.num_slots, s, j);
    float kf[4] = {0.0f, 0.0f, 0.0f, 0.0f}, vf[4] = {0.0f, 0.0f, 0.0f, 0.0f};
    float sk = 0.0f, sv = 0.0f;
    if (row >= 0) {
      const int64_t e = (row * nkv + g) * HD + 4 * lane, b = (row >> c.sb_shift) * nkv + g;
      codes_f32<KV>(*reinterpret_cast<const uint32_t*>(static_cast<const uint8_t*>(c.k) + e), kf);
      codes_f32<KV>(*reinterpret_cast<const uint32_t*>(static_cast<const uint8_t*>(c.v) + e), vf);
      sk = c.k_scale[b];
      sv = c.v_scale[b];
    }
    const float d = warp_sum(qv[0] * kf[0] + qv[1] * kf[1] + qv[2] * kf[2] + qv[3] * kf[3]);
    const float x = d * sk * scale_log2;
    const float m_new = fmaxf(m, x);
    const float alpha = exp2f(m - m_new), pr = exp2f(x - m_new);
    l = l * alpha + pr;
#pragma unroll
    for (int e = 0; e < 4; ++e) o[e] = o[e] * alpha + pr * sv * vf[e];
    m = m_new;
  }
  const float inv = l > 0.0f ? 1.0f / l : 0.0f;
#pragma unroll
  for (int e = 0; e < 4; ++e) out[at + e] = from_f<bf16>(o[e] * inv);
}

int launch_attn(const void* q, const Cache& c, const int32_t* cu_q, const int32_t* ctx, int n_seqs, int max_q, int nh,
                int nkv, int max_ctx, float scale, int window, int n_sink, void* out, int kv_dtype, cudaStream_t st) {
  const int64_t threads = int64_t(n_seqs) * max_q * nh * 32;
  const unsigned ctas = unsigned((threads + 127) / 128);
  if (kv_dtype == QW_I8)
    launch_pdl(attn_kv8_kernel<QW_I8>, ctas, 128, 0, st, static_cast<const bf16*>(q), c, cu_q, ctx, n_seqs, max_q, nh,
               nkv, max_ctx, scale * kLog2e, window, n_sink, static_cast<bf16*>(out));
  else
    launch_pdl(attn_kv8_kernel<QW_E4M3>, ctas, 128, 0, st, static_cast<const bf16*>(q), c, cu_q, ctx, n_seqs, max_q, nh,
               nkv, max_ctx, scale * kLog2e, window, n_sink, static_cast<bf16*>(out));
  return check_launch("attn_kv8_kernel");
}

// Checks shared by the two attention entry points.
int check_attention(const char* who, const void* k, const void* v, const float* ks, const float* vs, int64_t num_slots,
                    int scale_block, const int32_t* table, int max_blocks, int block_size, int n_seqs, int max_context,
                    int nh, int nkv, int head_dim, int window, int n_sink, int dtype, int kv_dtype) {
  if (dtype != QW_BF16) return set_error(QW_ERR_DTYPE, "%s: bf16 only", who);
  if (n_seqs < 0 || max_context < 0 || nh <= 0 || nkv <= 0 || window < 0 || n_sink < 0)
    return set_error(QW_ERR_INVALID_ARG, "%s: bad sizes", who);
  if (head_dim != HD || nh % nkv || nh / nkv > 16)
    return set_error(QW_ERR_SHAPE, "%s: needs head_dim 128 and nh a multiple of nkv, at most 16 times it", who);
  int rc = check_cache(who, k, v, ks, vs, num_slots, scale_block, kv_dtype);
  if (rc) return rc;
  rc = check_table(who, table, max_blocks, block_size, scale_block);
  if (rc) return rc;
  if (int64_t(max_context) > int64_t(max_blocks) * block_size)
    return set_error(QW_ERR_SHAPE, "%s: max_context %d > max_blocks x block_size", who, max_context);
  return QW_OK;
}

}  // namespace kv8
}  // namespace qw

using namespace qw;

extern "C" size_t qw_attention_decode_kv8_workspace_size(int B, int max_context, int n_heads, int n_kv_heads) {
  return B < 0 || max_context < 0 || n_heads <= 0 || n_kv_heads <= 0 ? 0 : kCounterBytes;
}

extern "C" int qw_attention_decode_kv8(const void* q, const void* k_cache, const void* v_cache, const float* k_scale,
                                       const float* v_scale, int64_t num_slots, int scale_block,
                                       const int32_t* context_lens, const int32_t* block_table, int max_blocks,
                                       int block_size, int B, int max_context, int n_heads, int n_kv_heads,
                                       int head_dim, float scale, int window, int n_sink, void* out, void* workspace,
                                       size_t workspace_bytes, int dtype, int kv_dtype, void* stream) {
  const char* who = "qw_attention_decode_kv8";
  const int rc = kv8::check_attention(who, k_cache, v_cache, k_scale, v_scale, num_slots, scale_block, block_table,
                                      max_blocks, block_size, B, max_context, n_heads, n_kv_heads, head_dim, window,
                                      n_sink, dtype, kv_dtype);
  if (rc) return rc;
  if (B == 0) return QW_OK;
  if (!q || !context_lens || !out) return set_error(QW_ERR_INVALID_ARG, "%s: null pointer", who);
  if (!kv8::aligned16(q) || !kv8::aligned16(out))
    return set_error(QW_ERR_INVALID_ARG, "%s: q and out must be 16-byte aligned", who);
  if (int64_t(B) * n_kv_heads > int64_t(kCounterBytes / sizeof(unsigned int)))
    return set_error(QW_ERR_SHAPE, "%s: %d sequences x %d kv heads exceed the counter area", who, B, n_kv_heads);
  const size_t need = qw_attention_decode_kv8_workspace_size(B, max_context, n_heads, n_kv_heads);
  if (!workspace || workspace_bytes < need)
    return set_error(QW_ERR_WORKSPACE, "%s: workspace of %zu bytes needed", who, need);
  const kv8::Cache c{k_cache, v_cache, k_scale, v_scale, num_slots, kv8::scale_shift(scale_block), block_table,
                     max_blocks, block_size};
  return kv8::launch_attn(q, c, nullptr, context_lens, B, 1, n_heads, n_kv_heads, max_context, scale, window, n_sink, out, kv_dtype,
                          static_cast<cudaStream_t>(stream));
}

extern "C" size_t qw_attention_prefill_kv8_workspace_size(int n_seqs, int64_t total_q, int max_seqlen_q,
                                                          int max_context, int n_heads, int n_kv_heads) {
  (void)n_seqs; (void)total_q; (void)max_seqlen_q; (void)max_context; (void)n_heads; (void)n_kv_heads;
  return 0;
}

extern "C" int qw_attention_prefill_kv8(const void* q, const void* k_cache, const void* v_cache, const float* k_scale,
                                        const float* v_scale, int64_t num_slots, int scale_block,
                                        const int32_t* cu_seqlens_q, const int32_t* context_lens,
                                        const int32_t* block_table, int max_blocks, int block_size, int n_seqs,
                                        int64_t total_q, int max_seqlen_q, int max_context, int n_heads,
                                        int n_kv_heads, int head_dim, float scale, int window, int n_sink, void* out,
                                        void* workspace, size_t workspace_bytes, int dtype, int kv_dtype,
                                        void* stream) {
  const char* who = "qw_attention_prefill_kv8";
  if (total_q < 0 || max_seqlen_q < 0) return set_error(QW_ERR_INVALID_ARG, "%s: bad sizes", who);
  const int rc = kv8::check_attention(who, k_cache, v_cache, k_scale, v_scale, num_slots, scale_block, block_table,
                                      max_blocks, block_size, n_seqs, max_context, n_heads, n_kv_heads, head_dim,
                                      window, n_sink, dtype, kv_dtype);
  if (rc) return rc;
  if (n_seqs == 0 || max_seqlen_q == 0 || total_q == 0) return QW_OK;
  if (!q || !cu_seqlens_q || !context_lens || !out) return set_error(QW_ERR_INVALID_ARG, "%s: null pointer", who);
  if (!kv8::aligned16(q) || !kv8::aligned16(out))
    return set_error(QW_ERR_INVALID_ARG, "%s: q and out must be 16-byte aligned", who);
  const size_t need =
      qw_attention_prefill_kv8_workspace_size(n_seqs, total_q, max_seqlen_q, max_context, n_heads, n_kv_heads);
  if (need > 0 && (!workspace || workspace_bytes < need))
    return set_error(QW_ERR_WORKSPACE, "%s: workspace of %zu bytes needed", who, need);
  const kv8::Cache c{k_cache, v_cache, k_scale, v_scale, num_slots, kv8::scale_shift(scale_block), block_table,
                     max_blocks, block_size};
  return kv8::launch_attn(q, c, cu_seqlens_q, context_lens, n_seqs, max_seqlen_q, n_heads, n_kv_heads, max_context, scale,
                          window, n_sink, out, kv_dtype, static_cast<cudaStream_t>(stream));
}

namespace qw {
unsigned int take_kv8_errors() {
  unsigned int v = 0, z = 0;
  cudaMemcpyFromSymbol(&v, kv8::g_kv8_error, sizeof(v));
  if (v) cudaMemcpyToSymbol(kv8::g_kv8_error, &z, sizeof(z));
  return v;
}
}  // namespace qw
