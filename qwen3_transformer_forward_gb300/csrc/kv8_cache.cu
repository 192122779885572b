// Writing and reading the 8-bit paged KV cache: QK-RMSNorm + RoPE + quantised
// append (qw_kv8_append) and rows back as values (qw_kv8_read).
#include <algorithm>

#include "kv8.cuh"

namespace qw {
namespace kv8 {

struct AppendArgs {
  const bf16* qkv;            // [T, tp * (nh/tp + 2 nkv/tp) * 128]
  int64_t T;
  int nh, nkv, tp;
  const int64_t* positions;   // [T]
  const float* cos_sin;       // [max_pos, 128]
  int64_t max_pos;
  const bf16* q_gamma;
  const bf16* k_gamma;
  float eps;
  const int32_t* cu_q;        // [n_seqs + 1], or null: one token per sequence
  const int32_t* ctx;         // [n_seqs]
  const int32_t* table;
  int max_blocks, block_size, n_seqs;
  uint8_t* k;
  uint8_t* v;
  float* k_scale;
  float* v_scale;
  int64_t num_slots;
  bf16* q_out;
  int32_t* err;
  int64_t kv_ctas;            // CTAs ahead of the q ones
};

__device__ __forceinline__ int seq_begin(const AppendArgs& a, int s) { return a.cu_q != nullptr ? a.cu_q[s] : s; }

// The sequence and the scale block of block task `t`: sequences in order, each
// with the blocks that its new tokens touch.  One warp scans the sequences 32
// at a time.  s = -1 when there are fewer tasks.
__device__ __forceinline__ void find_block(const AppendArgs& a, int64_t t, int sb, int& s_out, int& blk_out) {
  const int lane = threadIdx.x & 31;
  int64_t before = 0;
  s_out = -1;
  blk_out = 0;
  for (int s0 = 0; s0 < a.n_seqs; s0 += 32) {
    const int s = s0 + lane;
    int cnt = 0, b0 = 0;
    if (s < a.n_seqs) {
      const int lq = seq_begin(a, s + 1) - seq_begin(a, s), ctx = a.ctx[s];
      const int first = max(ctx - lq, 0);
      b0 = first / sb;
      cnt = lq > 0 && ctx > 0 ? (ctx - 1) / sb - b0 + 1 : 0;
    }
    int64_t upto = cnt;   // inclusive prefix sum
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int64_t y = __shfl_up_sync(0xffffffffu, upto, o);
      if (lane >= o) upto += y;
    }
    const bool here = t >= before + upto - cnt && t < before + upto;
    const unsigned m = __ballot_sync(0xffffffffu, here);
    if (m) {
      const int src = __ffs(m) - 1;
      s_out = s0 + src;
      blk_out = __shfl_sync(0xffffffffu, b0 + int(t - (before + upto - cnt)), src);
      return;
    }
    before += __shfl_sync(0xffffffffu, upto, 31);
  }
}

// One CTA per (scale block touched, kv head, K or V) with eight lanes per token
// of the block, then CTAs of eight lanes per (token, q head).  Lane `sub` owns
// elements 8 sub .. + 7 and 64 + 8 sub .. + 7 of its head, so RoPE pairs meet in
// one lane.  A block's tokens meet in one CTA because they share a scale: the
// block maximum is formed in shared memory and every value is quantised from
// the registers that it was computed in, so each input is read once.
template <int KV, int SB>
__global__ void __launch_bounds__(SB * 8) kv8_append_kernel(const AppendArgs a) {
  pdl_wait();      // inputs of this kernel are complete and visible
  pdl_trigger();   // only now may the next kernel start its prologue
  constexpr int HALF = 64, THREADS = SB * 8;
  const int sub = threadIdx.x & 7, grp = threadIdx.x >> 3, i0 = 8 * sub;
  const int nh_l = a.nh / a.tp, nkv_l = a.nkv / a.tp;
  const int64_t width_r = int64_t(nh_l + 2 * nkv_l) * HD, row_w = width_r * a.tp;

  // normed and roped head at src; `round_n`: the norm's output rounded to bf16
  auto norm_rope = [&](const bf16* src, const bf16* gamma, int64_t tok, bool round_n, float* y1, float* y2) {
    const int64_t pos = a.positions[tok];
    float x1[8], x2[8], g1[8], g2[8], c[8], sn[8];
    load16(src + i0, x1);
    load16(src + HALF + i0, x2);
    load16(gamma + i0, g1);
    load16(gamma + HALF + i0, g2);
    const bool pos_ok = pos >= 0 && pos < a.max_pos;
    const float* cs = a.cos_sin + (pos_ok ? pos : 0) * HD;
    *reinterpret_cast<float4*>(c) = *reinterpret_cast<const float4*>(cs + i0);
    *reinterpret_cast<float4*>(c + 4) = *reinterpret_cast<const float4*>(cs + i0 + 4);
    *reinterpret_cast<float4*>(sn) = *reinterpret_cast<const float4*>(cs + HALF + i0);
    *reinterpret_cast<float4*>(sn + 4) = *reinterpret_cast<const float4*>(cs + HALF + i0 + 4);
    const unsigned lanes = 0xffu << (threadIdx.x & 24);   // this token's eight lanes
    float ss = qk_ss8(x1, x2);
    ss = __fadd_rn(ss, __shfl_xor_sync(lanes, ss, 1));
    ss = __fadd_rn(ss, __shfl_xor_sync(lanes, ss, 2));
    ss = __fadd_rn(ss, __shfl_xor_sync(lanes, ss, 4));
    const float inv = qk_inv_rms(ss, a.eps);
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      if (round_n) {
        qk_rope_pair(x1[e], x2[e], inv, g1[e], g2[e], c[e], sn[e], pos_ok, y1[e], y2[e]);
      } else {
        const float n1 = __fmul_rn(__fmul_rn(x1[e], inv), g1[e]), n2 = __fmul_rn(__fmul_rn(x2[e], inv), g2[e]);
        y1[e] = pos_ok ? __fsub_rn(__fmul_rn(n1, c[e]), __fmul_rn(n2, sn[e])) : 0.0f;
        y2[e] = pos_ok ? __fadd_rn(__fmul_rn(n2, c[e]), __fmul_rn(n1, sn[e])) : 0.0f;
      }
    }
    return pos_ok;
  };

  if (blockIdx.x >= a.kv_ctas) {   // ---- q heads
    const int64_t unit = (int64_t(blockIdx.x) - a.kv_ctas) * (THREADS / 8) + grp;
    const int64_t tok = unit / a.nh;
    const int h = int(unit % a.nh);
    if (tok >= a.T || tok < seq_begin(a, 0) || tok >= seq_begin(a, a.n_seqs)) return;   // rows of no sequence
    float y1[8], y2[8];
    const bool pos_ok = norm_rope(a.qkv + tok * row_w + (h / nh_l) * width_r + int64_t(h % nh_l) * HD, a.q_gamma, tok,
                                  true, y1, y2);
    bf16* o = a.q_out + (tok * a.nh + h) * int64_t(HD);
    store16(o + i0, y1);
    store16(o + HALF + i0, y2);
    if (!pos_ok && sub == 0 && h == 0 && a.err != nullptr) atomicAdd(a.err, 1);
    return;
  }

  // ---- K or V of one kv head in one scale block
  const bool is_v = blockIdx.x & 1;
  const int64_t t = (int64_t(blockIdx.x) >> 1) / a.nkv;
  const int g = int((int64_t(blockIdx.x) >> 1) % a.nkv);
  int s, blk;
  find_block(a, t, SB, s, blk);   // every warp, the same answer
  if (s < 0) return;
  const int tok0 = seq_begin(a, s), lq = seq_begin(a, s + 1) - tok0, ctx = a.ctx[s];
  const int start = ctx - lq;                     // key position of the sequence's first new token (may be negative)
  const int p = blk * SB + grp;                   // this group's key position
  const int64_t row0 = row_of(a.table, a.max_blocks, a.block_size, a.num_slots, s, blk * SB);
  const int64_t tok = int64_t(tok0) + (p - start);
  const bool fresh = p >= start && p < ctx && tok >= 0 && tok < a.T;
  if (row0 < 0) {   // no page: nothing is stored
    if (fresh && !is_v && g == 0 && sub == 0 && a.err != nullptr) {
      const int64_t pos = a.positions[tok];
      if (pos >= 0 && pos < a.max_pos) atomicAdd(a.err, 1);   // (a bad position is counted with the q heads)
    }
    return;
  }
  float y1[8], y2[8];
#pragma unroll
  for (int e = 0; e < 8; ++e) y1[e] = y2[e] = 0.0f;
  float top = 0.0f;
  if (fresh) {
    const bf16* src = a.qkv + tok * row_w + (g / nkv_l) * width_r + int64_t(nh_l + (is_v ? nkv_l : 0) + g % nkv_l) * HD;
    if (is_v) {
      const int64_t pos = a.positions[tok];
      load16(src + i0, y1);
      load16(src + HALF + i0, y2);
      if (pos < 0 || pos >= a.max_pos)
#pragma unroll
        for (int e = 0; e < 8; ++e) y1[e] = y2[e] = 0.0f;
    } else {
      norm_rope(src, a.k_gamma, tok, false, y1, y2);
    }
#pragma unroll
    for (int e = 0; e < 8; ++e) {   // the largest finite magnitude
      const float u = fabsf(y1[e]), w = fabsf(y2[e]);
      top = fmaxf(top, u < INFINITY ? u : 0.0f);
      top = fmaxf(top, w < INFINITY ? w : 0.0f);
    }
  }
  __shared__ float s_top[THREADS / 32];
  top = warp_max(top);
  if ((threadIdx.x & 31) == 0) s_top[threadIdx.x >> 5] = top;
  float* scale = (is_v ? a.v_scale : a.k_scale) + (row0 / SB) * a.nkv + g;
  const bool held = start > blk * SB;             // tokens before the first new one
  const float was = held ? *scale : 0.0f;
  __syncthreads();                                // (every thread has read the old scale)
#pragma unroll
  for (int w = 0; w < THREADS / 32; ++w) top = fmaxf(top, s_top[w]);
  float cand = top / code_max<KV>();
  if (cand < kTinyScale) cand = 0.0f;
  const float now = fmaxf(was, cand);
  const float inv = now > 0.0f ? 1.0f / now : 0.0f;
  uint8_t* dst = (is_v ? a.v : a.k) + ((row0 + grp) * a.nkv + g) * int64_t(HD);
  if (fresh) {
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      y1[e] = __fmul_rn(y1[e], inv);
      y2[e] = __fmul_rn(y2[e], inv);
    }
    *reinterpret_cast<uint2*>(dst + i0) = make_uint2(quant4<KV>(y1), quant4<KV>(y1 + 4));
    *reinterpret_cast<uint2*>(dst + HALF + i0) = make_uint2(quant4<KV>(y2), quant4<KV>(y2 + 4));
  } else if (p < start && now > was) {            // an older token: its code in units of the new scale
    const float ratio = __fmul_rn(was, inv);
#pragma unroll
    for (int half = 0; half < 2; ++half) {
      uint2* w = reinterpret_cast<uint2*>(dst + half * HALF + i0);
      const uint2 c = *w;
      float f[8];
      codes_f32<KV>(c.x, f);
      codes_f32<KV>(c.y, f + 4);
#pragma unroll
      for (int e = 0; e < 8; ++e) f[e] = __fmul_rn(f[e], ratio);
      *w = make_uint2(quant4<KV>(f), quant4<KV>(f + 4));
    }
  }
  if (threadIdx.x == 0) *scale = now;
}

// Sixteen codes of K and of V per thread.
template <typename T, int KV>
__global__ void __launch_bounds__(256) kv8_read_kernel(const uint8_t* __restrict__ k, const uint8_t* __restrict__ v,
                                                       const float* __restrict__ ks, const float* __restrict__ vs,
                                                       int64_t num_slots, int sb_shift, int nkv,
                                                       const int64_t* __restrict__ rows, int64_t n,
                                                       T* __restrict__ k_out, T* __restrict__ v_out, int32_t* err) {
  pdl_wait();      // inputs of this kernel are complete and visible
  pdl_trigger();   // only now may the next kernel start its prologue
  const int64_t idx = int64_t(blockIdx.x) * blockDim.x + threadIdx.x;
  const int per_row = nkv * (HD / 16);
  if (idx >= n * per_row) return;
  const int64_t i = idx / per_row;
  const int c = int(idx % per_row), g = c / (HD / 16);
  const int64_t row = rows[i];
  const bool ok = row >= 0 && row < num_slots;
  if (!ok && row != -1 && c == 0 && err != nullptr) atomicAdd(err, 1);
  const int64_t at = (ok ? row : 0) * nkv * HD + 16 * c;
  const int64_t sc = ((ok ? row : 0) >> sb_shift) * nkv + g;
  uint4 a = make_uint4(0u, 0u, 0u, 0u), b = a;
  float sk = 0.0f, sv = 0.0f;
  if (ok && k_out != nullptr) {
    a = *reinterpret_cast<const uint4*>(k + at);
    sk = ks[sc];
  }
  if (ok && v_out != nullptr) {
    b = *reinterpret_cast<const uint4*>(v + at);
    sv = vs[sc];
  }
  auto put = [&](T* out, const uint4& w, float s) {
    float f[16];
    codes_f32<KV>(w.x, f);
    codes_f32<KV>(w.y, f + 4);
    codes_f32<KV>(w.z, f + 8);
    codes_f32<KV>(w.w, f + 12);
#pragma unroll
    for (int e = 0; e < 16; ++e) f[e] *= s;
    T* o = out + idx * 16;
#pragma unroll
    for (int e = 0; e < 16; e += V16<T>::N) store16(o + e, f + e);
  };
  if (k_out != nullptr) put(k_out, a, sk);
  if (v_out != nullptr) put(v_out, b, sv);
}

template <int KV>
int launch_append(const AppendArgs& a0, int scale_block, cudaStream_t st) {
  AppendArgs a = a0;
  // every touched block holds at least one new token, and a sequence with Lq of
  // them touches at most (Lq + sb - 2) / sb + 1 blocks
  const int64_t blocks = std::min(a.T, a.T / scale_block + 2 * int64_t(a.n_seqs));
  a.kv_ctas = blocks * a.nkv * 2;
  const int64_t per = scale_block;   // (token, q head) units of a CTA
  const int64_t ctas = a.kv_ctas + (a.T * a.nh + per - 1) / per;
  if (ctas > INT32_MAX) return set_error(QW_ERR_SHAPE, "qw_kv8_append: too many tokens");
  switch (scale_block) {
    case 16: launch_pdl(kv8_append_kernel<KV, 16>, unsigned(ctas), 128, 0, st, a); break;
    case 32: launch_pdl(kv8_append_kernel<KV, 32>, unsigned(ctas), 256, 0, st, a); break;
    default: launch_pdl(kv8_append_kernel<KV, 64>, unsigned(ctas), 512, 0, st, a); break;
  }
  return check_launch("kv8_append_kernel");
}

template <typename T, int KV>
int launch_read(const void* k, const void* v, const float* ks, const float* vs, int64_t num_slots, int scale_block,
                int nkv, const int64_t* rows, int64_t n, void* k_out, void* v_out, int32_t* err, cudaStream_t st) {
  const int64_t ctas = (n * nkv * (HD / 16) + 255) / 256;
  if (ctas > INT32_MAX) return set_error(QW_ERR_SHAPE, "qw_kv8_read: too many rows");
  launch_pdl(kv8_read_kernel<T, KV>, unsigned(ctas), 256, 0, st, static_cast<const uint8_t*>(k),
             static_cast<const uint8_t*>(v), ks, vs, num_slots, scale_shift(scale_block), nkv, rows, n,
             static_cast<T*>(k_out), static_cast<T*>(v_out), err);
  return check_launch("kv8_read_kernel");
}

}  // namespace kv8
}  // namespace qw

using namespace qw;

extern "C" int qw_kv8_append(const void* qkv, int64_t T, int n_heads, int n_kv_heads, int head_dim, int tp,
                             const int64_t* positions, const float* cos_sin, int64_t max_position, const void* q_gamma,
                             const void* k_gamma, float eps, const int32_t* cu_seqlens_q, const int32_t* context_lens,
                             const int32_t* block_table, int max_blocks, int block_size, int n_seqs, void* k_cache,
                             void* v_cache, float* k_scale, float* v_scale, int64_t num_slots, int scale_block,
                             void* q_out, int32_t* err_count, int dtype, int kv_dtype, void* stream) {
  const char* who = "qw_kv8_append";
  if (dtype != QW_BF16) return set_error(QW_ERR_DTYPE, "%s: bf16 only", who);
  if (T < 0 || n_seqs < 0 || n_heads <= 0 || n_kv_heads <= 0 || tp <= 0 || max_position <= 0)
    return set_error(QW_ERR_INVALID_ARG, "%s: bad sizes", who);
  if (head_dim != kv8::HD || n_heads % tp || n_kv_heads % tp)
    return set_error(QW_ERR_SHAPE, "%s: needs head_dim 128 and tp | nh, nkv", who);
  if (!cu_seqlens_q && T < n_seqs)
    return set_error(QW_ERR_SHAPE, "%s: %lld tokens for %d sequences of one token", who, (long long)T, n_seqs);
  int rc = kv8::check_cache(who, k_cache, v_cache, k_scale, v_scale, num_slots, scale_block, kv_dtype);
  if (rc) return rc;
  rc = kv8::check_table(who, block_table, max_blocks, block_size, scale_block);
  if (rc) return rc;
  if (T == 0 || n_seqs == 0) return QW_OK;
  if (!qkv || !positions || !cos_sin || !q_gamma || !k_gamma || !context_lens || !q_out)
    return set_error(QW_ERR_INVALID_ARG, "%s: null pointer", who);
  if (!kv8::aligned16(qkv) || !kv8::aligned16(cos_sin) || !kv8::aligned16(q_gamma) || !kv8::aligned16(k_gamma) ||
      !kv8::aligned16(q_out))
    return set_error(QW_ERR_INVALID_ARG, "%s: qkv, cos_sin, gammas and q_out must be 16-byte aligned", who);
  kv8::AppendArgs a;
  a.qkv = static_cast<const bf16*>(qkv);
  a.T = T;
  a.nh = n_heads;
  a.nkv = n_kv_heads;
  a.tp = tp;
  a.positions = positions;
  a.cos_sin = cos_sin;
  a.max_pos = max_position;
  a.q_gamma = static_cast<const bf16*>(q_gamma);
  a.k_gamma = static_cast<const bf16*>(k_gamma);
  a.eps = eps;
  a.cu_q = cu_seqlens_q;
  a.ctx = context_lens;
  a.table = block_table;
  a.max_blocks = max_blocks;
  a.block_size = block_size;
  a.n_seqs = n_seqs;
  a.k = static_cast<uint8_t*>(k_cache);
  a.v = static_cast<uint8_t*>(v_cache);
  a.k_scale = k_scale;
  a.v_scale = v_scale;
  a.num_slots = num_slots;
  a.q_out = static_cast<bf16*>(q_out);
  a.err = err_count;
  a.kv_ctas = 0;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  return kv_dtype == QW_I8 ? kv8::launch_append<QW_I8>(a, scale_block, st)
                           : kv8::launch_append<QW_E4M3>(a, scale_block, st);
}

extern "C" int qw_kv8_read(const void* k_cache, const void* v_cache, const float* k_scale, const float* v_scale,
                           int64_t num_slots, int scale_block, int n_kv_heads, int head_dim, const int64_t* rows,
                           int64_t n_rows, void* k_out, void* v_out, int32_t* err_count, int dtype, int kv_dtype,
                           void* stream) {
  const char* who = "qw_kv8_read";
  if (dtype != QW_BF16 && dtype != QW_F32) return set_error(QW_ERR_DTYPE, "%s: dtype %d", who, dtype);
  if (n_rows < 0 || n_kv_heads <= 0) return set_error(QW_ERR_INVALID_ARG, "%s: bad sizes", who);
  if (head_dim != kv8::HD) return set_error(QW_ERR_SHAPE, "%s: needs head_dim 128", who);
  const int rc = kv8::check_cache(who, k_cache, v_cache, k_scale, v_scale, num_slots, scale_block, kv_dtype);
  if (rc) return rc;
  if (n_rows == 0 || (!k_out && !v_out)) return QW_OK;
  if (!rows) return set_error(QW_ERR_INVALID_ARG, "%s: null rows", who);
  if (!kv8::aligned16(k_out) || !kv8::aligned16(v_out))
    return set_error(QW_ERR_INVALID_ARG, "%s: outputs must be 16-byte aligned", who);
  cudaStream_t st = static_cast<cudaStream_t>(stream);
#define QW_READ(TT, KV)                                                                                             \
  kv8::launch_read<TT, KV>(k_cache, v_cache, k_scale, v_scale, num_slots, scale_block, n_kv_heads, rows, n_rows, k_out, \
                           v_out, err_count, st)
  if (dtype == QW_BF16) return kv_dtype == QW_I8 ? QW_READ(bf16, QW_I8) : QW_READ(bf16, QW_E4M3);
  return kv_dtype == QW_I8 ? QW_READ(float, QW_I8) : QW_READ(float, QW_E4M3);
#undef QW_READ
}
